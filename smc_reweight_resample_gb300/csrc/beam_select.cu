// beam_select.cu -- the best continuations of every group's beams over the vocabulary.
//
// Candidate (beam i, token v) of a group has the score s_i + c z_iv - L_i with L_i = log sum_v exp(c z_iv), c = 1 / temperature; with
// the row's maximum m_i that is s_i + c (z_iv - m_i) - log S_i, S_i = sum_v exp(c (z_iv - m_i)).
// The M best of a group's N * V candidates are wanted, in the order of score, beam, token.
//
// One pass over the logits: a warp takes a chunk of 4 KB (eight 16-byte vectors a lane, loads back to back) and leaves its
// maximum, its sum of exp(c (z - maximum)) and the maxima of its eight sets (a set: the 32 lanes' vectors of one load, 512
// contiguous bytes). Nothing is selected on the way. Of ranges of tokens ordered by their maxima, ties by place, the first M
// hold the M best tokens: each of these M ranges has a token that comes before any token of a range behind them. So the last
// block of a group to finish
//   - adds up the beams' sums, which gives every score up to the beam's own constant,
//   - finds M (to 2 M) of the group's chunks, then M of those chunks' sets, by bisection on their maxima's scores,
//   - reads these sets again and keeps what is not below the last of them: a little more than M candidates,
//   - ranks them by counting.
// Scores are compared as double-floats (FP64 runs at two lanes a clock here), relative to the group's best one, in 64-bit keys
// whose order is theirs. Of one beam this order is exact, whatever its sum; between beams it is as good as the sums: hardware
// exponentials and float sums of 64 terms are off by at most 1.3e-6 (see kTol). Where two scores of different beams that decide
// anything are nearer than that, the block computes the beams' sums again in double-floats (1e-12) and selects anew.
#include "ops_launch.cuh"
#include "smcsd_launch.cuh"

namespace smcsd {

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamKeys = 4096;  // keys of a level in shared memory
constexpr int kBeamCands = 1024; // candidates that are ranked

// Bound on how far the scores of two beams may be off from one another with hardware exponentials. Of one sum, relative: the
// exponential 2^-22, its argument's two roundings at most 2^-23 (x 2^-x has its maximum 0.53 / ln 2 there), at most 7 + 8 + 5
// additions one after another 20 * 2^-24, the chunks' scale 2^-22 and their sum in 64 bits: 1.9e-6; two sums: 3.8e-6.
constexpr float kTol = 4.0e-6f;

// A score as an unsigned integer of the same order: the high float first, then the low one (of a normalised double-float). 0 is
// no score (minus infinity, NaN).
__device__ __forceinline__ uint32_t float_order(float f) {
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of_order(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(dd s) {
    if (!(s.hi > kNegInf) || !(s.hi < kPosInf)) return 0;
    return (uint64_t)float_order(s.hi + 0.0f) << 32 | float_order(s.lo + 0.0f);  // -0 is 0
}
__device__ __forceinline__ dd key_value(uint64_t k) { return dd{float_of_order((uint32_t)(k >> 32)), float_of_order((uint32_t)k)}; }
// c (z - m) + base, m being the row's maximum
__device__ __forceinline__ uint64_t score_key(const BeamParams& p, float z, float m, float2 base) {
    if (!(z > kNegInf)) return 0;
    return key_of(dd_add(dd_mul(two_sum(z, -m), dd{p.c_hi, p.c_lo}), dd{base.x, base.y}));
}

// Row r: its first vector begins `shift` elements before the row, at a multiple of 16 bytes.
template <int DT>
struct BeamRow {
    const char* at;  // first vector
    const char* row;
    int shift, V;
};
template <int DT>
__device__ __forceinline__ BeamRow<DT> beam_row(const BeamParams& p, long long r) {
    BeamRow<DT> b;
    b.row = static_cast<const char*>(p.logits) + r * p.row_stride * Geo<DT>::kBytes;
    const int off = (int)(reinterpret_cast<uintptr_t>(b.row) & 15u);
    b.at = b.row - off;
    b.shift = off / Geo<DT>::kBytes;
    b.V = p.V;
    return b;
}
__device__ __forceinline__ uint4 ld_vec(const char* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// Vector v of the row; tokens outside the row are -inf, and memory outside the row is not read.
template <int DT>
__device__ __forceinline__ uint4 beam_vec(const BeamRow<DT>& b, int v) {
    constexpr int PV = Geo<DT>::kPerVec;
    const long long e0 = (long long)v * PV - b.shift;
    if (e0 >= 0 && e0 + PV <= b.V) return ld_vec(b.at + 16ll * v);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = DT == 0 ? neg_inf_bits<0>() : neg_inf_bits<1>() * 0x10001u;
        if (DT == 0) {
            if (e0 + i >= 0 && e0 + i < b.V) w[i] = logit_bits<0>(b.row, e0 + i);
        } else {
            const long long e = e0 + 2 * i;
            if (e >= 0 && e < b.V) w[i] = (w[i] & 0xffff0000u) | logit_bits<1>(b.row, e);
            if (e + 1 >= 0 && e + 1 < b.V) w[i] = (w[i] & 0xffffu) | logit_bits<1>(b.row, e + 1) << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ void unpack(const uint4& x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == 0) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& x) {
    if (DT == 0)
        return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
    const uint32_t m = max_bf16x2(max_bf16x2(x.x, x.y), max_bf16x2(x.z, x.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
}
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One chunk of a row: its maximum, sum and set maxima. NaN and +inf show in the sum.
template <int DT>
__device__ __forceinline__ void beam_chunk(const BeamParams& p, const BeamRow<DT>& b, int chunk, float2* part, float* sets, int lane) {
    constexpr int PV = Geo<DT>::kPerVec;
    uint4 x[kBeamSets];
    const int v0 = chunk * kBeamSets * 32;
    const long long e0 = (long long)v0 * PV - b.shift;
    if (e0 >= 0 && e0 + kBeamSets * 32 * PV <= b.V) {
#pragma unroll
        for (int s = 0; s < kBeamSets; ++s) x[s] = ld_vec(b.at + 16ll * (v0 + s * 32 + lane));
    } else {
#pragma unroll
        for (int s = 0; s < kBeamSets; ++s) x[s] = beam_vec<DT>(b, v0 + s * 32 + lane);
    }
    float m = kNegInf, mine = kNegInf;
#pragma unroll
    for (int s = 0; s < kBeamSets; ++s) {
        const float a = warp_max(vec_max<DT>(x[s]));
        if (lane == s) mine = a;
        m = fmaxf(m, a);
    }
    float sum = 0.0f;
    if (m > kNegInf) {
#pragma unroll
        for (int s = 0; s < kBeamSets; ++s) {
            float f[PV];
            unpack<DT>(x[s], f);
#pragma unroll
            for (int i = 0; i < PV; ++i) f[i] = ex2_fast((f[i] - m) * p.c2);
#pragma unroll
            for (int o = PV / 2; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) f[i] += f[i + o];
            sum += f[0];
        }
        sum = warp_sum(sum);
    } else {
        // nothing but -inf, unless there are NaN, which the maxima pass over
        bool nan = false;
#pragma unroll
        for (int s = 0; s < kBeamSets; ++s) {
            float f[PV];
            unpack<DT>(x[s], f);
#pragma unroll
            for (int i = 0; i < PV; ++i) nan |= f[i] != f[i];
        }
        if (__any_sync(0xffffffffu, nan)) sum = __int_as_float(0x7fffffff);
    }
    if (lane < kBeamSets) sets[lane] = mine;
    if (lane == 0) *part = make_float2(m, sum);
}

struct BeamShared {
    double based[kBeamMostBeams];  // S_i, then s_i - log S_i: the beam's best score (of a finished beam s_i)
    float2 base[kBeamMostBeams];   // the same, relative to the group's best score
    float zmin[kBeamMostBeams];    // no candidate below this logit
    float zmax[kBeamMostBeams];    // the row's maximum
    int live[kBeamMostBeams];      // beams whose rows are read
    int over[kBeamMostBeams];      // finished beams
    int nlive, nover;
    int list1[2 * kBeamMost], list2[2 * kBeamMost], order[kBeamMost + 1];
    int count, last;
    double ref;
    unsigned long long reduce, fixed[2];
    union {
        uint64_t keys[kBeamKeys];
        struct {
            uint64_t key[kBeamCands];
            uint64_t at[kBeamCands];  // beam, token
        } cand;
    };
};
static_assert(sizeof(BeamShared) <= 48 * 1024, "static shared memory");

__device__ __forceinline__ int count_from(const uint64_t* keys, int n, uint64_t from) {
    int c = 0;
    for (int i = threadIdx.x; i - (int)threadIdx.x < n; i += kBeamThreads) c += __syncthreads_count(i < n && keys[i] >= from);
    return c;
}
// What is kept of n keys: those above K, and those equal to K before place I; between M and `most` of them, the first in the
// order of keys and places (all that are not 0 if they are no more than `most`).
struct Cut {
    uint64_t K;
    int I;
};
__device__ __forceinline__ bool kept(const Cut& c, uint64_t key, int i) { return key > c.K || (key == c.K && i < c.I); }
__device__ Cut find_cut(const uint64_t* keys, int n, int M, int most) {
    if (count_from(keys, n, 1) <= most) return Cut{0, 0};
    uint64_t lo = 1, hi = ~0ull;  // more than `most` from lo on, fewer than M from hi on
    while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        const int c = count_from(keys, n, mid);
        if (c > most)
            lo = mid;
        else if (c < M)
            hi = mid;
        else
            return Cut{mid, n};
    }
    // many are equal to lo: the first places of them
    int a = 0, b = n;
    while (b - a > 1) {
        const int mid = a + (b - a) / 2;
        int c = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x < n; i += kBeamThreads) c += __syncthreads_count(i < n && kept(Cut{lo, mid}, keys[i], i));
        if (c < M)
            a = mid;
        else if (c > most)
            b = mid;
        else
            return Cut{lo, mid};
    }
    return Cut{lo, b};
}

// The places of what is kept, ascending, in `list`; returns how many.
__device__ int gather_kept(BeamShared& s, const uint64_t* keys, int n, const Cut& cut, int* list) {
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBeamThreads)
        if (kept(cut, keys[i], i)) {
            const int k = atomicAdd(&s.count, 1);
            if (k < 2 * kBeamMost) list[k] = i;
        }
    __syncthreads();
    const int got = min(s.count, 2 * kBeamMost);
    // by counting: the list is short
    int mine[2 * kBeamMost / kBeamThreads], rank[2 * kBeamMost / kBeamThreads];
#pragma unroll
    for (int t = 0; t < 2 * kBeamMost / kBeamThreads; ++t) {
        const int i = threadIdx.x + t * kBeamThreads;
        rank[t] = 0;
        if (i < got) {
            mine[t] = list[i];
            for (int j = 0; j < got; ++j) rank[t] += list[j] < mine[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2 * kBeamMost / kBeamThreads; ++t)
        if ((int)threadIdx.x + t * kBeamThreads < got) list[rank[t]] = mine[t];
    __syncthreads();
    return got;
}

// Sum of exp(c (z - m)) over row b by the whole block: every term from double-floats, rounded to a multiple of 2^-56 and added up
// in integers, so that rows with the same logits have the same sum however they lie in memory. Off by at most 2^-57 a term and
// 1e-13 of it.
template <int DT>
__device__ double precise_sum(const BeamParams& p, BeamShared& s, const BeamRow<DT>& b, float m) {
    constexpr int PV = Geo<DT>::kPerVec;
    const int vecs = (int)(((long long)b.V + b.shift + PV - 1) / PV);
    unsigned __int128 acc = 0;
    for (int v = threadIdx.x; v < vecs; v += kBeamThreads) {
        float f[PV];
        unpack<DT>(beam_vec<DT>(b, v), f);
#pragma unroll 1
        for (int i = 0; i < PV; ++i) {
            const dd x = dd_mul(two_sum(f[i], -m), dd{p.c_hi, p.c_lo});
            if (!(x.hi > -42.0f)) continue;  // below 2^-60
            const ddx e = exp_split(x, p.T);
            const float u = pow2i(e.n + 56);
            acc += (unsigned long long)(__float2ll_rn(e.hi * u) + __float2ll_rn(e.lo * u));
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) s.fixed[0] = s.fixed[1] = 0;
    __syncthreads();
    // in units of 2^-56 and 2^-24: both stay below 2^63 with 2^31 terms
    atomicAdd(&s.fixed[0], (unsigned long long)acc & 0xffffffffull);
    atomicAdd(&s.fixed[1], (unsigned long long)(acc >> 32));
    __syncthreads();
    return ldexp((double)s.fixed[1], -24) + ldexp((double)s.fixed[0], -56);
}

// Calls f(key, beam, token) for every token of the sets in list2 whose logit is not below its beam's zmin.
template <int DT, typename F>
__device__ __forceinline__ void scan_sets(const BeamParams& p, BeamShared& s, int g, int n2, F&& f) {
    constexpr int PV = Geo<DT>::kPerVec;
    const int lane = threadIdx.x & 31, per = p.cpr * kBeamSets;
    for (int i = threadIdx.x >> 5; i < n2; i += kBeamWarps) {
        const int set = s.list2[i], l = set / per, beam = s.live[l], v = (set - l * per) * 32 + lane;
        const BeamRow<DT> b = beam_row<DT>(p, (long long)g * p.N + beam);
        float z[PV];
        unpack<DT>(beam_vec<DT>(b, v), z);
        const float zmin = s.zmin[beam], m = s.zmax[beam];
        const float2 base = s.base[beam];
#pragma unroll
        for (int e = 0; e < PV; ++e)
            if (z[e] >= zmin) {
                const uint64_t key = score_key(p, z[e], m, base);
                if (key) f(key, beam, (int)((long long)v * PV + e - b.shift));
            }
    }
}

// Adds up one count a thread.
__device__ __forceinline__ unsigned long long block_total(BeamShared& s, unsigned mine) {
    __syncthreads();
    if (threadIdx.x == 0) s.reduce = 0;
    __syncthreads();
    const unsigned w = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0 && w) atomicAdd(&s.reduce, (unsigned long long)w);
    __syncthreads();
    return s.reduce;
}

// Candidates by beam and token; kEnded stands for the token of a finished beam.
constexpr int kEnded = -1;
__device__ __forceinline__ uint64_t place_of(int beam, int token) { return (uint64_t)(uint32_t)beam << 32 | (uint32_t)token; }
__device__ __forceinline__ float start_score(const BeamParams& p, int g, int beam) {
    return p.scores ? __ldg(p.scores + (long long)g * p.N + beam) : 0.0f;
}

// Fills s.cand with the candidates that can be among the first M; returns how many, and in `floor` the key below which
// candidates were left out (0: none were).
template <int DT>
__device__ int collect(const BeamParams& p, BeamShared& s, int g, uint64_t& floor) {
    const int M = p.M, most = min(2 * M, M + 64), nlive = s.nlive;
    const float2* part = ws_ptr<const float2>(p.ws, p.part) + (long long)g * p.N * p.cpr;
    const float* sets = ws_ptr<const float>(p.ws, p.sets) + (long long)g * p.N * p.cpr * kBeamSets;
    const int n = nlive * p.cpr;
    uint64_t* keys = n <= kBeamKeys ? s.keys : ws_ptr<uint64_t>(p.ws, p.keys) + (long long)g * p.N * p.cpr;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const int l = i / p.cpr, beam = s.live[l];
        keys[i] = score_key(p, __ldcg(part + beam * p.cpr + (i - l * p.cpr)).x, s.zmax[beam], s.base[beam]);
    }
    __syncthreads();
    const Cut c1 = find_cut(keys, n, M, most);
    const int n1 = gather_kept(s, keys, n, c1, s.list1);
    for (int i = threadIdx.x; i < n1 * kBeamSets; i += kBeamThreads) {
        const int chunk = s.list1[i / kBeamSets], l = chunk / p.cpr, beam = s.live[l];
        s.keys[i] = score_key(p, __ldcg(sets + ((long long)beam * p.cpr + (chunk - l * p.cpr)) * kBeamSets + i % kBeamSets),
                              s.zmax[beam], s.base[beam]);
    }
    __syncthreads();
    const Cut c2 = find_cut(s.keys, n1 * kBeamSets, M, most);
    const int n2 = gather_kept(s, s.keys, n1 * kBeamSets, c2, s.list2);
    // places in list1 to sets of the group's live beams
    for (int i = threadIdx.x; i < n2; i += kBeamThreads) s.list2[i] = s.list1[s.list2[i] / kBeamSets] * kBeamSets + s.list2[i] % kBeamSets;
    floor = c1.K > c2.K ? c1.K : c2.K;
    // the floor as a logit of each live beam, lowered by more than its rounding
    const float at = floor ? key_value(floor).hi : kNegInf;
    for (int l = threadIdx.x; l < nlive; l += kBeamThreads) {
        const int beam = s.live[l];
        const float b = s.base[beam].x, m = s.zmax[beam], z = m + (at - b) / p.c_hi;
        s.zmin[beam] = floor ? z - (fabsf(m) + (fabsf(at) + fabsf(b)) / p.c_hi) * 1e-6f - 1e-35f : -3.402823466e38f;
    }
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    const int room = kBeamCands - s.nover;
    uint64_t K = floor, I = ~0ull;  // kept: keys above K, and those equal to K up to place I
    scan_sets<DT>(p, s, g, n2, [&](uint64_t key, int beam, int token) {
        if (key >= K) {
            const int k = atomicAdd(&s.count, 1);
            if (k < room) s.cand.key[k] = key, s.cand.at[k] = place_of(beam, token);
        }
    });
    __syncthreads();
    if (s.count > room) {
        // many tokens next to one another in the order: bisection over the tokens themselves
        uint64_t lo = K, hi = ~0ull;
        bool found = false;
        auto total = [&](uint64_t k, uint64_t i) {
            unsigned mine = 0;
            scan_sets<DT>(p, s, g, n2, [&](uint64_t key, int beam, int token) { mine += key > k || (key == k && place_of(beam, token) <= i); });
            return block_total(s, mine);
        };
        while (hi - lo > 1 && !found) {
            const uint64_t mid = lo + (hi - lo) / 2;
            const unsigned long long c = total(mid, ~0ull);
            if (c > (unsigned)room)
                lo = mid;
            else if (c < (unsigned)M)
                hi = mid;
            else
                K = mid, found = true;
        }
        if (!found) {
            K = lo;
            uint64_t a = 0, b = place_of(p.N, 0);
            I = b;
            while (b - a > 1) {
                const uint64_t mid = a + (b - a) / 2;
                const unsigned long long c = total(K, mid);
                if (c < (unsigned)M) {
                    a = mid;
                } else {
                    b = I = mid;
                    if (c <= (unsigned)room) break;
                }
            }
        }
        floor = K;
        __syncthreads();
        if (threadIdx.x == 0) s.count = 0;
        __syncthreads();
        scan_sets<DT>(p, s, g, n2, [&](uint64_t key, int beam, int token) {
            if (key > K || (key == K && place_of(beam, token) <= I)) {
                const int k = atomicAdd(&s.count, 1);
                if (k < room) s.cand.key[k] = key, s.cand.at[k] = place_of(beam, token);
            }
        });
        __syncthreads();
    }
    const int got = min(s.count, room);
    for (int i = threadIdx.x; i < s.nover; i += kBeamThreads) {
        const int beam = s.over[i];
        s.cand.key[got + i] = key_of(dd{s.base[beam].x, s.base[beam].y});
        s.cand.at[got + i] = place_of(beam, kEnded);
    }
    __syncthreads();
    return got + s.nover;
}

// Ranks the candidates: s.order holds the first M (and one more, if there is one). Whether scores of different beams that
// decide about this order are nearer than the sums are good for.
__device__ bool rank_and_doubt(const BeamParams& p, BeamShared& s, int n, uint64_t floor) {
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const uint64_t key = s.cand.key[i], at = s.cand.at[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s.cand.key[j] > key || (s.cand.key[j] == key && s.cand.at[j] < at);
        if (rank <= p.M) s.order[rank] = i;
    }
    __syncthreads();
    bool doubt = false;
    auto near = [&](int i, int j) {
        const uint64_t a = s.cand.at[i], b = s.cand.at[j];
        if (a >> 32 == b >> 32 || ((int)(uint32_t)a == kEnded && (int)(uint32_t)b == kEnded)) return false;  // of one beam; exact
        const dd d = dd_sub(key_value(s.cand.key[i]), key_value(s.cand.key[j]));
        return fabsf(d.hi) <= kTol;
    };
    const int m = min(p.M, n);
    for (int r = threadIdx.x; r < m && r + 1 < n; r += kBeamThreads) doubt |= near(s.order[r], s.order[r + 1]);
    if (n > p.M) {  // what is next to the last one, on either side, in any beam
        const int last = s.order[p.M - 1];
        for (int i = threadIdx.x; i < n; i += kBeamThreads) doubt |= near(i, last);
    }
    if (floor && n >= p.M && s.nlive + s.nover > 1) {  // and what was left out
        // (a bisection's key need not be one of a double-float: its high half is as near as that half's last place)
        const float f = key_value(floor).hi;
        doubt |= key_value(s.cand.key[s.order[p.M - 1]]).hi - f <= kTol + 2.4e-7f * fabsf(f);
    }
    return __syncthreads_or(doubt);
}

// The group's selection, by the last block of the group.
template <int DT>
__device__ void beam_finish(const BeamParams& p, BeamShared& s, int g) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2* part = ws_ptr<const float2>(p.ws, p.part) + (long long)g * p.N * p.cpr;
    // a warp a beam: maximum and sum of its chunks
    for (int l = warp; l < s.nlive; l += kBeamWarps) {
        const float2* q = part + (long long)s.live[l] * p.cpr;
        float m = kNegInf;
        for (int k = lane; k < p.cpr; k += 32) m = fmaxf(m, __ldcg(q + k).x);
        m = warp_max(m);
        double sum = 0.0;
        for (int k = lane; k < p.cpr; k += 32) {
            const float2 x = __ldcg(q + k);
            if (x.x > kNegInf)
                sum += (double)(x.y * exp2f((x.x - m) * p.c2));
            else if (x.y != x.y)
                sum += (double)x.y;
        }
        sum = warp_sum_d(sum);
        if (lane == 0) {
            s.zmax[s.live[l]] = m;
            s.based[s.live[l]] = sum;
        }
    }
    __syncthreads();
    bool precise = false;
    int n;
    for (;;) {
        // the beams' constants: scores are c (z - m) + base
        for (int l = threadIdx.x; l < s.nlive; l += kBeamThreads) {
            const int beam = s.live[l];
            const double sum = s.based[beam];
            const float m = s.zmax[beam];
            double base = (double)kNegInf;
            if (!(sum < (double)kPosInf) || m == kPosInf)
                raise_error(p.ws, kErrNonfinite);
            else if (sum > 0.0)
                base = (double)start_score(p, g, beam) - log(sum);
            s.based[beam] = base;
        }
        for (int i = threadIdx.x; i < s.nover; i += kBeamThreads) s.based[s.over[i]] = (double)start_score(p, g, s.over[i]);
        __syncthreads();
        if (warp == 0) {  // the best score, which all others are taken relative to
            double best = (double)kNegInf;
            for (int l = lane; l < s.nlive; l += 32) best = fmax(best, s.based[s.live[l]]);
            for (int i = lane; i < s.nover; i += 32) best = fmax(best, s.based[s.over[i]]);
            best = warp_max_d(best);
            if (lane == 0) s.ref = best;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < s.nlive + s.nover; i += kBeamThreads) {
            const int beam = i < s.nlive ? s.live[i] : s.over[i - s.nlive];
            const double b = s.based[beam] - s.ref;
            const float hi = (float)b;
            s.base[beam] = b > (double)kNegInf ? make_float2(hi, (float)(b - (double)hi)) : make_float2(kNegInf, 0.0f);
        }
        __syncthreads();
        uint64_t floor;
        n = collect<DT>(p, s, g, floor);
        const bool doubt = rank_and_doubt(p, s, n, floor);
        if (!doubt || precise) break;
        precise = true;
        for (int l = 0; l < s.nlive; ++l) {
            const int beam = s.live[l];
            const float m = s.zmax[beam];
            const bool whole = s.based[beam] > (double)kNegInf;
            const double sum = whole ? precise_sum<DT>(p, s, beam_row<DT>(p, (long long)g * p.N + beam), m) : 0.0;
            __syncthreads();
            if (threadIdx.x == 0) s.based[beam] = sum;
        }
        __syncthreads();
    }
    for (int r = threadIdx.x; r < p.M; r += kBeamThreads) {
        int token = p.pad, beam = 0, over = 1;
        float score = kNegInf;
        if (r < n && s.cand.key[s.order[r]]) {
            const uint64_t at = s.cand.at[s.order[r]];
            beam = (int)(at >> 32);
            const long long row = (long long)g * p.N + beam;
            if ((int)(uint32_t)at == kEnded) {
                score = start_score(p, g, beam);
            } else {
                token = (int)(uint32_t)at;
                const float z = logit_at<DT>(beam_row<DT>(p, row).row, token);
                score = (float)(s.based[beam] + p.c * ((double)z - (double)s.zmax[beam]));
                over = p.eos >= 0 && token == p.eos;
            }
        }
        const long long o = (long long)g * p.M + r;
        p.tokens[o] = token;
        p.ancestors[o] = beam;
        p.out_scores[o] = score;
        if (p.out_finished) p.out_finished[o] = over;
    }
}

template <int DT>
__global__ void __launch_bounds__(kBeamThreads, 2) beam_kernel(const __grid_constant__ BeamParams p) {
    __shared__ BeamShared s;
    const int g = blockIdx.x / p.blocks, b = blockIdx.x - g * p.blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {  // beams in order: those whose rows are read, and the finished ones
        int live = 0, over = 0;
        for (int i0 = 0; i0 < p.N; i0 += 32) {
            const int i = i0 + lane;
            const long long row = (long long)g * p.N + i;
            const float score = i < p.N ? start_score(p, g, i) : kNegInf;
            if (!(score < kPosInf) && b == 0) raise_error(p.ws, kErrNonfinite);
            const bool some = score > kNegInf && score < kPosInf;
            const bool ended = some && p.finished && __ldg(p.finished + row);
            const unsigned l = __ballot_sync(0xffffffffu, some && !ended), o = __ballot_sync(0xffffffffu, ended);
            const unsigned below = (1u << lane) - 1u;
            if (some && !ended) s.live[live + __popc(l & below)] = i;
            if (ended) s.over[over + __popc(o & below)] = i;
            live += __popc(l);
            over += __popc(o);
        }
        if (lane == 0) s.nlive = live, s.nover = over;
    }
    __syncthreads();
    float2* part = ws_ptr<float2>(p.ws, p.part);
    float* sets = ws_ptr<float>(p.ws, p.sets);
    const int items = s.nlive * p.cpr;
    for (int i = b * kBeamWarps + warp; i < items; i += p.blocks * kBeamWarps) {
        const int l = i / p.cpr, chunk = i - l * p.cpr;
        const long long row = (long long)g * p.N + s.live[l], at = row * p.cpr + chunk;
        beam_chunk<DT>(p, beam_row<DT>(p, row), chunk, part + at, sets + at * kBeamSets, lane);
    }
    __syncthreads();
    if (p.blocks > 1) {
        if (threadIdx.x == 0) {
            unsigned* count = ws_ptr<unsigned>(p.ws, p.count) + g;
            s.last = atom_add_release(count, 1u) == (unsigned)p.blocks - 1u;
            if (s.last) {
                fence_acquire();
                atomicExch(count, 0u);
            }
        }
        __syncthreads();
        if (!s.last) return;
    }
    beam_finish<DT>(p, s, g);
}

cudaError_t launch_beam(const BeamParams& p0, int dtype, cudaStream_t st) {
    BeamParams p = p0;
    // a chunk for each warp, as long as all blocks run at the same time
    const long long chunks = (long long)p.N * p.cpr, want = (chunks + kBeamWarps - 1) / kBeamWarps;
    const long long fit = 2ll * device_sm_count() / p.G;
    p.blocks = (int)(want < fit ? want : fit);
    if (p.blocks < 1) p.blocks = 1;
    const unsigned grid = (unsigned)p.G * (unsigned)p.blocks;
    if (dtype == 0)
        beam_kernel<0><<<grid, kBeamThreads, 0, st>>>(p);
    else
        beam_kernel<1><<<grid, kBeamThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace smcsd
