// distill_loss.cu -- a draft's loss against a teacher's top logits, and its gradient, in one pass over the logits.
//
// q = softmax(c z) over the vocabulary, c = 1 / temperature; p the teacher's probabilities of the row's listed tokens, p_r what they
// leave to the rest (0 where the list is taken for everything):
//   loss = sum_k p_k (log p_k - log q_k) + p_r (log p_r - log q_r),     q_r = sum of q over the tokens that are not listed;
//   dloss / dz_v = c (P q_v - p_v) for a listed v,  c q_v (P - p_r / q_r) for others,     P = sum p + p_r.
// For the gradient a cluster of blocks holds a row in shared memory: read once, added up, and written from there when the blocks'
// sums have met in the cluster's shared memories. For the loss alone rows are read to registers. Where there is a rest, the listed
// tokens are left out of the sum, so that q_r is a sum and no difference.
#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "ops_launch.cuh"
#include "smcsd_launch.cuh"

namespace cg = cooperative_groups;

namespace smcsd {

constexpr int kDistillThreads = 256, kDistillMoreThreads = 384, kDistillMostThreads = 512;
// Vectors of a block that holds its share, as long as sixteen blocks are enough for a row: in blocks of 256 threads, six to an SM; and in
// blocks of 384, four to an SM, where that makes a row's blocks half as many and there are two for each SM all the same. Us with the
// larger shares / the smaller: 4096 rows of 43000 bf16 130 / 143, of 90000 276 / 297, of 24000 76.9 / 77.6; 300 of 43000 11.4 / 14.1, of
// 24000 9.1 / 8.8; 40 of 90000 8.3 / 7.7.
constexpr int kDistillStaged = 2560, kDistillMore = 3328;
constexpr int kDistillRead = 16384;   // of a block that reads it, where rows are many
static_assert(kDistillThreads >= kDistillMostTokens, "a thread for each listed token");

__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int DT>
struct Elem;
template <>
struct Elem<0> {
    using T = uint32_t;
};
template <>
struct Elem<1> {
    using T = unsigned short;
};
template <int DT>
__device__ __forceinline__ uint32_t round_to(float f) {
    if (DT == 0) return __float_as_uint(f);
    unsigned short r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
}
// Maxima that pass over NaN: of words of the type, and of a word's halves.
template <int DT>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    uint32_t r;
    if (DT == 0)
        r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ float word_value(uint32_t a) {
    return DT == 0 ? __uint_as_float(a) : fmaxf(bf16_lo(a), bf16_hi(a));
}

// A sum of exp(c (z - m)) and its reference m. A reference of -inf goes with a sum of 0, or of NaN.
struct Mass {
    float m, s;
};
__device__ __forceinline__ float rescale(float from, float to, float c2) { return from > kNegInf ? exp2_fast((from - to) * c2) : 1.0f; }
__device__ __forceinline__ Mass warp_mass(Mass a, float c2) {
    const float m = warp_max(a.m);
    return Mass{m, warp_sum(a.s * rescale(a.m, m, c2))};
}
__device__ __forceinline__ Mass join(Mass a, Mass b, float c2) {
    const float m = fmaxf(a.m, b.m);
    return Mass{m, a.s * rescale(a.m, m, c2) + b.s * rescale(b.m, m, c2)};
}
// The same mass relative to about its logarithm, where the reference is far below that: a sum of up to 2^113 would make the gradient's
// factor a subnormal, or 0, for small weights. The factor between the two is good to 2^-23 (c2 (from - to) as a double-float).
__device__ __forceinline__ Mass centred(Mass a, float c2) {
    if (!(a.s > 16777216.0f && a.s < kPosInf)) return a;
    const float m = a.m + log2f(a.s) / c2;
    const dd d = two_sum(a.m, -m);
    const float t = f_mul(d.hi, c2), n = rintf(t);
    if (!(fabsf(t) < 126.0f)) return a;  // logits next to the end of float32's range
    return Mass{m, a.s * exp2f(n) * exp2f(f_add(f_sub(t, n), f_add(f_fma(d.hi, c2, -t), f_mul(d.lo, c2))))};
}
// Two masses each of up to 16 entries, on every lane of the calling warp.
struct Masses {
    Mass a, b;
};
__device__ __forceinline__ Masses join_lanes(const float4* q, int n, float c2) {
    const int lane = threadIdx.x & 31;
    const float4 x = lane < n ? q[lane] : make_float4(kNegInf, 0.0f, kNegInf, 0.0f);
    const float a = warp_max(x.x), b = warp_max(x.z);
    float sa = x.y * rescale(x.x, a, c2), sb = x.w * rescale(x.z, b, c2);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    return Masses{Mass{a, __shfl_sync(0xffffffffu, sa, 0)}, Mass{b, __shfl_sync(0xffffffffu, sb, 0)}};
}

// What the blocks of a cluster tell one another: stores to another block's shared memory that count on its barrier as they land, so
// that nothing but their landing is waited for (a barrier of the cluster waits for all earlier memory operations too: 200 us for 196 at
// 2048 x 128256, 101 for 94 at 4096 x 32000).
__device__ __forceinline__ uint32_t shared_address(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t in_block(uint32_t address, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(address), "r"(rank));
    return r;
}
__device__ __forceinline__ void tell(uint32_t at, float4 x, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at), "f"(x.x), "f"(x.y),
                 "f"(x.z), "f"(x.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tell_bits(uint32_t at, uint32_t x, uint32_t bar) {
    asm volatile("red.async.relaxed.cluster.shared::cluster.mbarrier::complete_tx::bytes.add.u32 [%0], %1, [%2];" ::"r"(at), "r"(x), "r"(bar) : "memory");
}
__device__ __forceinline__ void told_init(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool told(uint32_t bar) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar)
        : "memory");
    return ok != 0;
}
constexpr unsigned long long kToldNs = 2000000000ull;  // longest wait
__device__ __forceinline__ bool wait_told(uint32_t bar) {
#ifdef SMCSD_IMPATIENT
    if (cg::this_cluster().block_rank() & 1) return false;  // a test's build: every second block gives up at once
#endif
    if (told(bar)) return true;
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    while (!told(bar)) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > kToldNs) return false;
    }
    return true;
}

struct DistillShared {
    alignas(8) unsigned long long bar;  // what the other blocks tell this one
    alignas(16) int token[kDistillMostTokens];
    union {
        unsigned seen[kDistillMostTokens];  // a table of bits, then
        float p[kDistillMostTokens];
    };
    float z[kDistillMostTokens];    // in the first block: the listed tokens' logits
    float4 part[kDistillMostCtas];       // of each block: the rest's mass, the listed tokens' mass
    float4 q[kDistillMostThreads / 32];  // of each warp: the same
    float4 row;                          // the row's mass, the factor of the gradient and the reference that it goes with
    float a[kDistillMostTokens / 32], b[kDistillMostTokens / 32];
    dd d[kDistillMostTokens / 32];
    float rest, mass;
    int repeats, late;
};
// A block that has given up waiting (its context may have been off the GPU meanwhile) may still be told something, in shared memory that must
// not be another block's by then. All its threads stay until the cluster's others have come here too or left, who have told it all
// by then, and until that has landed.
__device__ __forceinline__ void stay(const DistillShared& s, uint32_t bar) {
    if (!s.late) return;
    cg::this_cluster().sync();  // whoever has left is not waited for
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        if (told(bar)) break;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < kToldNs);
}

// Maximum, or sum, over the list's entries, one of each thread of the block's first `warps` warps, which alone call these.
__device__ __forceinline__ void list_sync(int warps) { asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory"); }
__device__ __forceinline__ float list_max(DistillShared& s, float a, int warps) {
    a = warp_max(a);
    if (warps == 1) return a;
    if ((threadIdx.x & 31) == 0) s.a[threadIdx.x >> 5] = a;
    list_sync(warps);
    for (int w = 0; w < warps; ++w) a = fmaxf(a, s.a[w]);
    return a;
}
__device__ __forceinline__ float list_sum(DistillShared& s, float a, int warps) {
    a = warp_sum(a);
    if (warps == 1) return a;
    if ((threadIdx.x & 31) == 0) s.b[threadIdx.x >> 5] = a;
    list_sync(warps);
    a = s.b[0];
    for (int w = 1; w < warps; ++w) a += s.b[w];
    return a;
}
__device__ __forceinline__ dd list_sum_dd(DistillShared& s, float v, int warps) {
    dd a = warp_sum_dd(dd{v, 0.0f});
    if (warps == 1) return a;
    if ((threadIdx.x & 31) == 0) s.d[threadIdx.x >> 5] = a;
    list_sync(warps);
    a = s.d[0];
    for (int w = 1; w < warps; ++w) a = dd_add(a, s.d[w]);
    return a;
}

// This block's share of a row: n of the row's aligned vectors, the first of which begins at the row's element `e0`. It may begin
// before the row (the row's first vector) and end behind it (its last).
template <int DT>
struct Share {
    const char* at;  // first vector
    int n, e0, V;
    __device__ Share(const DistillParams& p, int r, int rank) {
        constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes;
        const char* row = static_cast<const char*>(after_wait(p.logits)) + (long long)r * p.row_stride * B;
        const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / B;
        const int first = rank * p.vecs, all = (p.V + shift + PV - 1) / PV - first;
        V = p.V;
        n = all < 0 ? 0 : all < p.vecs ? all : p.vecs;
        e0 = first * PV - shift;
        at = row + (long long)e0 * B;
    }
    // vectors that lie in the row whole: from whole_from() to whole_to() - 1; the first and the last one may not
    __device__ int whole_from() const { return e0 < 0 && n > 0 ? 1 : 0; }
    __device__ int whole_to() const { return n > 0 && e0 + n * Geo<DT>::kPerVec > V ? n - 1 : n; }
};

// Whether one of the warp's tokens, of those with `check`, stands in the list more than once. Of more than 32, tokens meet in a table of
// bits, and one that finds its bit set is looked for in the list by its warp. (Each thread going through the list took 40 us more for 2048 rows
// with 128 tokens each, 140 with 256.)
__device__ __forceinline__ bool list_repeats(int token, bool check, DistillShared& s, int warps) {
    const int lane = threadIdx.x & 31;
    if (warps == 1) return __any_sync(0xffffffffu, __popc(__match_any_sync(0xffffffffu, check ? token : -1 - lane)) > 1);
    const unsigned h = (unsigned)token * 0x9e3779b1u >> 19, bit = 1u << (h & 31);
    unsigned again = __ballot_sync(0xffffffffu, check && (atomicOr(s.seen + (h >> 5), bit) & bit));
    for (; again; again &= again - 1) {
        const int t = __shfl_sync(0xffffffffu, token, __ffs(again) - 1);
        int n = 0;
        for (int k = 0; k < 32 * warps; k += 32) n += __popc(__ballot_sync(0xffffffffu, s.token[k + lane] == t));
        if (n > 1) return true;
    }
    return false;
}

// A thread's entry of the row's list. All threads call this; whether the list has any mass.
struct Entry {
    int token;
    float value;
    // the logarithm of the teacher's probability; in the token's first place the probability of all its entries
    float logp, listed;
    bool first;
};
__device__ __forceinline__ bool list_entry(const DistillParams& p, DistillShared& s, int r, Entry& e) {
    const int tid = threadIdx.x;
    e.token = -1;
    e.value = kNegInf;
    if (tid < p.K) {
        e.token = __ldg(after_wait(p.tokens) + (long long)r * p.K + tid);
        e.value = __ldg(after_wait(p.values) + (long long)r * p.K + tid);
        if (e.token < 0 || e.token >= p.V) {
            if (e.token != -1) raise_error(p.ws, kErrRange);
            e.token = -1;
            e.value = kNegInf;
        } else if (!(e.value < kPosInf)) {
            raise_error(p.ws, kErrNonfinite);
        }
    }
    if (tid < kDistillMostTokens) s.token[tid] = e.token, s.seen[tid] = 0;
    if (tid == 0) s.repeats = 0, s.late = 0;
    return __syncthreads_or(e.value > kNegInf);
}
// The teacher's probabilities, by the warps with entries; p_r and the sum of all too.
__device__ __forceinline__ void list_teacher(const DistillParams& p, DistillShared& s, Entry& e, bool check, int lists) {
    const int tid = threadIdx.x;
    float rest = 0.0f, mass = 1.0f, prob;
    if (p.rest) {
        e.logp = e.value;
        prob = e.value > kNegInf ? expf(e.value) : 0.0f;
        const dd sum = list_sum_dd(s, prob, lists);
        // A list of all that has mass leaves nothing, but for roundings: of the values (half a step of each, 2^-24 of the list's entropy, which is
        // 5.6 at most) and of their exponentials (2^-23). A rest of that kind would make the loss infinite where q leaves nothing either.
        rest = dd_add(dd{1.0f, 0.0f}, dd_neg(sum)).hi;
        if (!(rest >= 4.76837158e-7f)) rest = 0.0f;  // 2^-21
        mass = rest > 0.0f ? 1.0f : sum.hi;
    } else {
        const float top = list_max(s, e.value, lists);
        const float x = e.value > kNegInf ? expf(e.value - top) : 0.0f;
        const dd sum = list_sum_dd(s, x, lists);
        e.logp = e.value - top - logf(sum.hi);
        prob = x / sum.hi;
    }
    e.listed = prob;
    if (list_repeats(e.token, check, s, lists) && (tid & 31) == 0) s.repeats = 1;
    list_sync(lists);
    s.p[tid] = prob;
    if (tid == 0) s.rest = rest, s.mass = mass;
    if (!s.repeats) return;
    // a token that is listed several times: its first place stands for all of them
    list_sync(lists);
    if (e.token < 0) return;
    e.listed = 0.0f;
    for (int k = p.K - 1; k >= 0; --k)
        if (s.token[k] == e.token) {
            e.listed += s.p[k];
            e.first = k == tid;
        }
}
// The loss, by the first block's warps with entries, from the row's mass and the rest's.
__device__ __forceinline__ void list_loss(const DistillParams& p, DistillShared& s, const Entry& e, int lists, float z, Mass all, Mass R, int r) {
    const float ls = logf(all.s);
    float term = 0.0f;
    const float prob = s.p[threadIdx.x], rest = s.rest;
    if (prob > 0.0f) {
        const float away = z - all.m, logq = away * p.c - ls;
        // a token masked with the lowest value: log q may lie below float32's range though its share of the loss does not
        term = logq == kNegInf && away > kNegInf ? -(prob * p.c) * away : prob * (e.logp - logq);
    }
    if (threadIdx.x == 0 && rest > 0.0f) term += rest * (logf(rest) - (logf(R.s) + (R.m - all.m) * p.c - ls));
    const float loss = list_sum(s, term, lists);
    if (threadIdx.x == 0) p.loss[r] = loss;
}
__device__ __forceinline__ Mass token_mass(const Entry& e, float z) {
    return e.first ? Mass{z, z > kNegInf ? 1.0f : z != z ? z : 0.0f} : Mass{kNegInf, 0.0f};
}

// Elements of a vector one by one: f(e, bits) for those from `lo` to `hi` - 1.
template <int DT, typename F>
__device__ __forceinline__ void each_element(const uint4& x, int lo, int hi, F&& f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < Geo<DT>::kPerVec; ++e)
        if (e >= lo && e < hi) f(e, DT == 0 ? w[e & 3] : (w[(e >> 1) & 3] >> (16 * (e & 1))) & 0xffffu);
}

// The share on its way to shared memory, its whole vectors as they are, of the others the elements that lie in the row.
template <int DT, int TH>
__device__ __forceinline__ void fetch(const Share<DT>& h, uint4* to) {
    constexpr int PV = Geo<DT>::kPerVec;
    using T = typename Elem<DT>::T;
    const int from = h.whole_from(), upto = h.whole_to();
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    for (int i = from + threadIdx.x; i < upto; i += TH) copy16_async(at + 16u * i, h.at + 16ll * i);
    if (threadIdx.x < 2 * PV) {  // a thread for each element of the first and the last vector
        const int i = threadIdx.x < PV ? 0 : h.n - 1, e = threadIdx.x & (PV - 1), v = h.e0 + i * PV + e;
        if (i < h.n && i >= 0 && (i < from || i >= upto))
            reinterpret_cast<T*>(to + i)[e] = (T)(v >= 0 && v < h.V ? logit_bits<DT>(h.at, (long long)i * PV + e) : neg_inf_bits<DT>());
    }
}

__device__ __forceinline__ void st_vec(char* p, const uint4& x) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Writes f(i), a vector, for every vector i of the share to the row `out` of the gradient.
template <int DT, int TH, typename F>
__device__ __forceinline__ void write_share(const Share<DT>& h, char* out, F&& f) {
    constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes;
    using T = typename Elem<DT>::T;
    char* to = out + (long long)h.e0 * B;
    const bool alike = (reinterpret_cast<uintptr_t>(to) & 15u) == 0;
    const int from = alike ? h.whole_from() : h.n, upto = alike ? h.whole_to() : h.n;
#pragma unroll 1
    for (int i = from + threadIdx.x; i < upto; i += TH) st_vec(to + 16ll * i, f(i));
    if (from == 0 && upto == h.n) return;
    // the first and the last vector, or all of a row that lies otherwise than the logits'
    for (int i = threadIdx.x; i < h.n; i += TH) {
        if (i >= from && i < upto) continue;
        const int v = h.e0 + i * PV;
        each_element<DT>(f(i), v < 0 ? -v : 0, v + PV > h.V ? h.V - v : PV, [&](int e, uint32_t bits) { reinterpret_cast<T*>(to)[(long long)i * PV + e] = (T)bits; });
    }
}

// Shares of up to 40 KB: six blocks of 256 threads in an SM, each at another point of its row, so that loads, sums and stores overlap.
// 2048 rows of 128256 bf16 with 64 tokens each take 191 us, 155 at the copy rate; of that 20 are the sums (issue; measured by leaving them out),
// the rest is a row's structure: list, copies, the meeting of eight blocks, writing. DRAM reads and writes each row once. With 256 tokens
// 221: probabilities of eight warps in every block.
template <int DT, int TH>
__global__ void __launch_bounds__(TH, TH == kDistillThreads ? 6 : TH == kDistillMoreThreads ? 4 : 3) distill_kernel(const __grid_constant__ DistillParams p) {
    constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes;
    using T = typename Elem<DT>::T;
    extern __shared__ uint4 s_row[];
    __shared__ DistillShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = p.ctas, rank = (int)cl.block_rank(), tid = threadIdx.x;
    const int r = blockIdx.x / C;
    // Each block of a row tells all of them its masses, and the first one the listed tokens' logits (whose bits add up, those of the others
    // being 0); it leaves when all have told it theirs. How much is told does not depend on the list, of which blocks read different
    // ones where it changes meanwhile.
    const uint32_t bar = shared_address(&s.bar);
    const bool tell_z = p.loss && tid < p.K;
    if (rank == 0 && tid < kDistillMostTokens) s.z[tid] = 0.0f;
    if (tid == 0 && C > 1) told_init(bar, 16 * C + (rank == 0 && p.loss ? 4 * p.K * C : 0));
    auto started = cl.barrier_arrive();  // the other blocks may be told something once all have come here
    const auto meet = [&](float4 own) {  // by the first warp
        if (C == 1) {
            if (tid == 0) s.part[0] = own;
            __syncwarp();
            return;
        }
        if (tid < C) tell(in_block(shared_address(&s.part[rank]), tid), own, in_block(bar, tid));
        if (!wait_told(bar)) {
            s.late = 1;
            raise_error(p.ws, kErrTimeout);  // no counters are left behind
        }
    };

    griddep_wait();
    const Share<DT> h(p, r, rank);
    Entry e{};
    const bool some = list_entry(p, s, r, e);
    const int token = e.token;
    e.first = token >= 0;
    const float weight = p.weight ? __ldg(after_wait(p.weight) + r) : 1.0f;
    char* out = static_cast<char*>(p.grad) + (long long)r * p.grad_stride * B;

    if (!some || (weight == 0.0f && !p.loss)) {
        cl.barrier_wait(std::move(started));
        if (tell_z && C > 1) tell_bits(in_block(shared_address(&s.z[tid]), 0), 0, in_block(bar, 0));
        if (tid < 32) meet(make_float4(kNegInf, 0.0f, kNegInf, 0.0f));
        write_share<DT, TH>(h, out, [](int) { return make_uint4(0, 0, 0, 0); });
        if (rank == 0 && tid == 0 && p.loss) p.loss[r] = 0.0f;
        __syncthreads();
        stay(s, bar);
        return;
    }
    fetch<DT, TH>(h, s_row);
    // meanwhile the teacher's probabilities
    const int lists = (p.K + 31) / 32;  // warps with entries
    const bool lister = tid < 32 * lists;
    const int at = token - h.e0;
    const bool mine = token >= 0 && at >= 0 && at < h.n * PV;
    if (lister) list_teacher(p, s, e, mine, lists);
    T* elems = reinterpret_cast<T*>(s_row);
    float z = kNegInf;
    copies_done();
    // a thread has copied the vectors that it adds up itself, but for a first or last one that does not lie in the row whole
    if (p.rest || h.whole_from() > 0 || h.whole_to() < h.n) __syncthreads();
    if (p.rest) {  // the listed tokens are taken out of the share
        if (mine) z = bits_to_float<DT>((uint32_t)elems[at]);
        if (lister) list_sync(lists);
        if (mine) elems[at] = (T)neg_inf_bits<DT>();
        __syncthreads();
    }

    // the share's mass: each thread relative to its first vector's maximum, unless a later one is so much larger (or the first
    // one is masked) that the sum says little; then to its own maximum
    const f32x2 c2 = pair(p.c2, p.c2);
    const auto mass_of = [&](float m) {
        const float m0 = m > kNegInf ? -m : 0.0f;  // -inf alone adds up to 0, NaN to NaN
        const f32x2 m2 = pair(m0, m0);
        f32x2 sum[Vec<DT>::kPairs];
#pragma unroll
        for (int k = 0; k < Vec<DT>::kPairs; ++k) sum[k] = pair(0.0f, 0.0f);
#pragma unroll 1
        for (int i = tid; i < h.n; i += TH) {
            const Vec<DT> v(s_row[i]);
#pragma unroll
            for (int k = 0; k < Vec<DT>::kPairs; ++k) sum[k] = add2(sum[k], exp2_2(mul2(add2(v.x[k], m2), c2)));
        }
#pragma unroll
        for (int k = 1; k < Vec<DT>::kPairs; ++k) sum[0] = add2(sum[0], sum[k]);
        float lo, hi;
        halves(sum[0], lo, hi);
        return Mass{m, lo + hi};
    };
    Mass a{kNegInf, 0.0f};
    if (tid < h.n) {
        const uint4 x = s_row[tid];
        uint32_t top = word_max<DT>(word_max<DT>(x.x, x.y), word_max<DT>(x.z, x.w));
        for (bool whole = false;; whole = true) {
            a = mass_of(word_value<DT>(top));
            if (whole || (a.m > kNegInf && a.s < 1.2676506e30f)) break;  // 2^100
            for (int i = tid; i < h.n; i += TH) {
                const uint4 y = s_row[i];
                top = word_max<DT>(top, word_max<DT>(word_max<DT>(y.x, y.y), word_max<DT>(y.z, y.w)));
            }
        }
    }
    a = warp_mass(a, p.c2);
    Mass b{kNegInf, 0.0f};
    if (lister && p.rest) {
        if (mine) b = token_mass(e, z);
        b = warp_mass(b, p.c2);
    }
    if ((tid & 31) == 0) s.q[tid >> 5] = make_float4(a.m, a.s, b.m, b.s);
    cl.barrier_wait(std::move(started));
    __syncthreads();
    if (mine && !p.rest) z = bits_to_float<DT>((uint32_t)elems[at]);
    if (C == 1) {
        if (mine) s.z[tid] = z;
    } else if (tell_z) {
        tell_bits(in_block(shared_address(&s.z[tid]), 0), mine ? __float_as_uint(z) : 0u, in_block(bar, 0));
    }
    if (tid < 32) {
        const Masses q = join_lanes(s.q, TH / 32, p.c2);
        meet(make_float4(q.a.m, q.a.s, q.b.m, q.b.s));
    }

    // the row's mass, by one warp; without a rest all of it is in R
    const float wc = weight * p.c;
    if (tid < 32) {
        const Masses row = join_lanes(s.part, C, p.c2);
        const Mass all = centred(p.rest ? join(row.a, row.b, p.c2) : row.a, p.c2), R = p.rest ? centred(row.a, p.c2) : all;
        if (tid == 0) {
            // the rest relative to its own maximum; one without mass (all -inf) gets no gradient
            float scale = 0.0f;
            if (R.m > kNegInf) scale = p.rest ? wc * (s.mass * exp2f((R.m - all.m) * p.c2) / all.s - s.rest / R.s) : wc / all.s;
            s.row = make_float4(all.m, all.s, scale, R.m > kNegInf ? R.m : 0.0f);
            s.q[0].x = R.m, s.q[0].y = R.s;
            if (rank == 0 && !(all.s > 0.0f && all.s < kPosInf && all.m < kPosInf)) raise_error(p.ws, kErrNonfinite);
        }
    }
    __syncthreads();
    const float4 row = s.row;
    const Mass all{row.x, row.y};
    if (rank == 0 && lister && p.loss) list_loss(p, s, e, lists, s.z[tid], all, Mass{s.q[0].x, s.q[0].y}, r);
    const f32x2 m2 = pair(-row.w, -row.w), scale2 = pair(row.z, row.z);
    write_share<DT, TH>(h, out, [&](int i) {
        Vec<DT> v(s_row[i]);
#pragma unroll
        for (int k = 0; k < Vec<DT>::kPairs; ++k) v.x[k] = mul2(exp2_2(mul2(add2(v.x[k], m2), c2)), scale2);
        return v.packed();
    });
    __syncthreads();  // the listed tokens' places have been written as part of the rest
    if (mine && e.first) {
        const float q = exp2f((z - all.m) * p.c2) / all.s;
        reinterpret_cast<T*>(out)[token] = (T)round_to<DT>(wc * (s.mass * q - e.listed));
    }
    stay(s, bar);
}

// ------------------------------------------------------------------------------------------
// the loss alone: no share is held, so that shares may be large and a row's meeting comes seldom. 640 rows of 151936 float32 take 75 us,
// 57 at the copy rate (113 with the kernel above).
// ------------------------------------------------------------------------------------------

__device__ __forceinline__ uint4 ld_once(const char* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// Vector i of the share where a part of it lies outside the row: -inf there.
template <int DT>
__device__ __forceinline__ uint4 ragged_vec(const Share<DT>& h, int i) {
    constexpr int PV = Geo<DT>::kPerVec;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = DT == 0 ? neg_inf_bits<0>() : neg_inf_bits<1>() * 0x10001u;
#pragma unroll
    for (int e = 0; e < PV; ++e) {
        const int v = h.e0 + i * PV + e;
        if (v < 0 || v >= h.V) continue;
        const uint32_t bits = logit_bits<DT>(h.at, (long long)i * PV + e);
        if (DT == 0)
            w[e & 3] = bits;
        else
            w[(e >> 1) & 3] = e & 1 ? (w[(e >> 1) & 3] & 0xffffu) | bits << 16 : (w[(e >> 1) & 3] & 0xffff0000u) | bits;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Calls f(i, vector i) for this thread's vectors of the share, kEach of them on the way together.
template <int DT, int kEach, typename F>
__device__ __forceinline__ void each_vec(const Share<DT>& h, F&& f) {
    const int from = h.whole_from(), upto = h.whole_to();
    int i = from + threadIdx.x;
    const char* at = h.at + 16ll * i;
    for (; i < upto; i += kEach * kDistillThreads, at += 16 * kEach * kDistillThreads) {
        uint4 x[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (i + k * kDistillThreads < upto) x[k] = ld_once(at + 16 * k * kDistillThreads);
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (i + k * kDistillThreads < upto) f(i + k * kDistillThreads, x[k]);
    }
    // a first and a last vector that do not lie in the row whole
    if (threadIdx.x == 0 && from > 0) f(0, ragged_vec<DT>(h, 0));
    if (threadIdx.x == 1 && h.n - 1 >= upto && h.n - 1 >= from) f(h.n - 1, ragged_vec<DT>(h, h.n - 1));
}

template <int DT>
__global__ void __launch_bounds__(kDistillThreads, 6) distill_loss_kernel(const __grid_constant__ DistillParams p) {
    constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes, kEach = 4, kWarps = kDistillThreads / 32;
    extern __shared__ uint32_t s_listed[];  // where there is a rest: a bit for each element of the share, set if it is listed
    __shared__ DistillShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = p.ctas, rank = (int)cl.block_rank(), tid = threadIdx.x;
    const int r = blockIdx.x / C;
    auto started = cl.barrier_arrive();
    griddep_wait();
    const Share<DT> h(p, r, rank);
    if (p.rest)
        for (int i = tid; i < (h.n * PV + 31) / 32; i += kDistillThreads) s_listed[i] = 0;
    Entry e{};
    const bool some = list_entry(p, s, r, e);
    if (!some) {
        cl.barrier_wait(std::move(started));
        if (rank == 0 && tid == 0) p.loss[r] = 0.0f;
        cl.sync();  // every block stays for the last meeting, whatever list it has read
        return;
    }
    e.first = e.token >= 0;
    float z = kNegInf;  // of all shares: with a rest every block needs the listed tokens' mass, without one the first the loss
    if (e.token >= 0 && (p.rest || rank == 0))
        z = logit_at<DT>(static_cast<const char*>(after_wait(p.logits)) + (long long)r * p.row_stride * B, e.token);
    if (p.rest) {
        const int at = e.token - h.e0;
        if (e.token >= 0 && at >= 0 && at < h.n * PV) atomicOr(s_listed + (at >> 5), 1u << (at & 31));
        __syncthreads();
    }
    const auto unlisted = [&](int i, uint4 x) {  // -inf in the listed tokens' places
        if (p.rest) {
            const unsigned bits = reinterpret_cast<const unsigned char*>(s_listed)[i * PV >> 3] >> (i * PV & 7);
            if (bits & ((1u << PV) - 1u)) {
                const auto hide = [&](uint32_t w, unsigned b) {
                    if (DT == 0) return b & 1u ? neg_inf_bits<0>() : w;
                    return (b & 1u ? neg_inf_bits<1>() : w & 0xffffu) | (b & 2u ? neg_inf_bits<1>() << 16 : w & 0xffff0000u);
                };
                constexpr int kStep = PV / 4;
                x = make_uint4(hide(x.x, bits), hide(x.y, bits >> kStep), hide(x.z, bits >> (2 * kStep)), hide(x.w, bits >> (3 * kStep)));
            }
        }
        return x;
    };
    const auto top_of = [](const uint4& x) { return word_max<DT>(word_max<DT>(x.x, x.y), word_max<DT>(x.z, x.w)); };
    // as in the other kernel: relative to the first vector's maximum, or if that says little to the thread's own
    const f32x2 c2 = pair(p.c2, p.c2);
    uint32_t top = DT == 0 ? neg_inf_bits<0>() : neg_inf_bits<1>() * 0x10001u;
    if (tid < h.n) top = top_of(unlisted(tid, tid >= h.whole_from() && tid < h.whole_to() ? ld_once(h.at + 16ll * tid) : ragged_vec<DT>(h, tid)));
    Mass a{kNegInf, 0.0f};
#pragma unroll 1
    for (bool whole = false;; whole = true) {
        a.m = word_value<DT>(top);
        const float m0 = a.m > kNegInf ? -a.m : 0.0f;
        const f32x2 m2 = pair(m0, m0);
        f32x2 sum[Vec<DT>::kPairs];
#pragma unroll
        for (int k = 0; k < Vec<DT>::kPairs; ++k) sum[k] = pair(0.0f, 0.0f);
        each_vec<DT, kEach>(h, [&](int i, const uint4& x) {
            const Vec<DT> v(unlisted(i, x));
#pragma unroll
            for (int k = 0; k < Vec<DT>::kPairs; ++k) sum[k] = add2(sum[k], exp2_2(mul2(add2(v.x[k], m2), c2)));
        });
#pragma unroll
        for (int k = 1; k < Vec<DT>::kPairs; ++k) sum[0] = add2(sum[0], sum[k]);
        float lo, hi;
        halves(sum[0], lo, hi);
        a.s = lo + hi;
        if (whole || (a.m > kNegInf && a.s < 1.2676506e30f)) break;  // 2^100
        each_vec<DT, 1>(h, [&](int i, const uint4& x) { top = word_max<DT>(top, top_of(unlisted(i, x))); });
    }
    a = warp_mass(a, p.c2);
    const int lists = (p.K + 31) / 32;
    const bool lister = tid < 32 * lists;
    Mass b{kNegInf, 0.0f};
    if (lister) {
        if (rank == 0) list_teacher(p, s, e, e.token >= 0, lists);
        if (p.rest && rank == 0) b = warp_mass(token_mass(e, z), p.c2);
    }
    if ((tid & 31) == 0) s.q[tid >> 5] = make_float4(a.m, a.s, b.m, b.s);
    cl.barrier_wait(std::move(started));
    __syncthreads();
    if (tid < 32) {
        const Masses q = join_lanes(s.q, kWarps, p.c2);
        if (tid == 0) *cl.map_shared_rank(&s.part[rank], 0) = make_float4(q.a.m, q.a.s, q.b.m, q.b.s);
    }
    cl.sync();
    if (rank == 0 && lister) {
        const Masses row = join_lanes(s.part, C, p.c2);
        const Mass R = row.a, all = p.rest ? join(R, row.b, p.c2) : R;
        if (tid == 0 && !(all.s > 0.0f && all.s < kPosInf && all.m < kPosInf)) raise_error(p.ws, kErrNonfinite);
        list_loss(p, s, e, lists, z, all, R, r);
    }
}

// ------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------

template <typename F>
static cudaError_t launch_rows(F kernel, const DistillParams& p, int threads, size_t shared, cudaStream_t st) {
    cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), shared);
    if (e == cudaSuccess && p.ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
    }
    return launch_waiting(kernel, dim3((unsigned)((long long)p.R * p.ctas)), threads, shared, p.ctas, st, p);
}

template <int DT>
static cudaError_t launch_distill_as(DistillParams p, cudaStream_t st) {
    const long long vecs = ((long long)p.V * Geo<DT>::kBytes + 30) / 16;
    p.ctas = 1;
    if (p.grad) {
        while (p.ctas < kDistillMostCtas && vecs > p.ctas * (long long)kDistillStaged) {
            if (vecs <= p.ctas * (long long)kDistillMore && (long long)p.R * p.ctas >= 2ll * device_sm_count()) break;
            p.ctas *= 2;
        }
        p.vecs = (int)((vecs + p.ctas - 1) / p.ctas);
        const size_t shared = 16 * (size_t)p.vecs;
        if (p.vecs <= kDistillStaged) return launch_rows(distill_kernel<DT, kDistillThreads>, p, kDistillThreads, shared, st);
        if (p.vecs <= kDistillMore) return launch_rows(distill_kernel<DT, kDistillMoreThreads>, p, kDistillMoreThreads, shared, st);
        return launch_rows(distill_kernel<DT, kDistillMostThreads>, p, kDistillMostThreads, shared, st);
    }
    while (p.ctas < kDistillMostCtas && vecs > p.ctas * (long long)kDistillRead) p.ctas *= 2;
    // smaller shares where rows are few, for three turns of the blocks that run at a time
    while (p.ctas < kDistillMostCtas && vecs > p.ctas * 1024ll && (long long)p.R * p.ctas < 15ll * device_sm_count()) p.ctas *= 2;
    p.vecs = (int)((vecs + p.ctas - 1) / p.ctas);
    return launch_rows(distill_loss_kernel<DT>, p, kDistillThreads, p.rest ? (size_t)p.vecs * Geo<DT>::kPerVec / 8 + 4 : 0, st);
}

cudaError_t launch_distill(const DistillParams& p, int dtype, cudaStream_t st) {
    return dtype == 0 ? launch_distill_as<0>(p, st) : launch_distill_as<1>(p, st);
}

}  // namespace smcsd
