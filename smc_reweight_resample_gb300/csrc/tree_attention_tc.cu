// tree_attention_tc.cu -- attention of drafted tokens over a paged bf16 cache on the tensor cores.
//
// A row is a node and one of the query heads that share a key/value head. One block per SM walks its
// share of the line of key tiles (attn_plan.cuh); a tile is 128 keys.
//   warp 8     brings the pages of each tile into a ring of shared-memory stages (TMA, 128-byte swizzle):
//              keys, values, keys, values, ...
//   warp 9     issues the products: S = Q K^T (128 rows x 128 keys, sums in tensor memory) and
//              O += P V with P read from tensor memory
//   (warps 10 and 11 idle: registers are handed over by fours)
//   warps 0-7  two groups of four, one thread per row: maximum, exponentials, sum, and P (bf16) written
//              over S
// The groups are two streams that take turns on the tensor core: while one does its exponentials the
// products of the other run. With more than 128 rows in a unit the streams are two blocks of 128 rows
// over the same tiles; with fewer they are the even and the odd tiles of the same rows, joined at the
// end. A unit of few rows is bound by the bytes of its keys and values (one tile of 64 KB takes 1.5 us of
// an SM's share of memory, its products of 128 padded rows 0.5 us), one of many rows by the products
// and the exponentials.
//
// Softmax. With z = scale2 q.k (in units of log 2), a row keeps a reference m, l = sum exp2(z - m) and
// O = sum exp2(z - m) V. The reference moves (and O is rescaled) only when the maximum has grown by more
// than 8, so weights stay below 2^8: sums are in float32, P has bf16's 8 bits at any scale. l sums the
// weights before they are rounded. Rounding P to bf16 is what lets the second product run at bf16 rate;
// it is off by 2^-9 of each weight on average signs, less than the rounding of the result.
#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_plan.cuh"
#include "smcsd_launch.cuh"

namespace smcsd {

namespace {

constexpr int kTcThreads = 384;
constexpr int kTile = 128;       // keys of a tile, rows of a block
constexpr int kHalf = 128 * 128; // bytes of 128 rows of 64 bf16
constexpr unsigned long long kTcWaitNs = 2000000000ull;

template <int D>
struct TcGeo {
    static constexpr int kHalves = D / 64;
    static constexpr int kStage = kHalves * kHalf;         // one tile of keys or of values
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kSmem = 1024 + 2 * kStage + kStages * kStage;  // alignment, two blocks of q, the ring
};

// ---- instructions ----

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// both operands in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// the first operand in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void ld32(uint32_t addr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Shared-memory operand of a product: 128-byte swizzle. Rows along the sum's dimension (K-major): groups of
// 8 rows 1024 bytes apart. Rows along the output's dimension (the values: a key's 64 columns in a row):
// groups of 8 keys 1024 bytes apart, blocks of 64 columns kHalf apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(kHalf >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// Instruction: float32 sums, bf16 operands, 128 rows, n columns, second operand's rows along n if mn
constexpr uint32_t instruction(int n, int mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)mn << 16) | ((uint32_t)(n / 8) << 17) | ((128u / 16) << 24);
}

struct __align__(8) TcShared {
    uint64_t full[10], empty[10];  // ring
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint32_t tmem;
    int abort;
    int poison;  // a NaN or infinity among the values of the piece's nodes
};

// the eight warps of the rows
__device__ __forceinline__ void rows_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

struct Ctl {
    void* ws;
    int* abort;
};
// Waits are bounded: after about 2 s the error is recorded and every later wait of the block returns.
__device__ __forceinline__ void wait_slow(const Ctl& c, uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = now_ns();
    while (!mbar_try(bar, parity)) {
        if (*reinterpret_cast<volatile int*>(c.abort)) return;
        if (now_ns() - t0 > kTcWaitNs) {
            raise_error(c.ws, kErrTimeout);
            *reinterpret_cast<volatile int*>(c.abort) = 1;
            return;
        }
    }
}
// one thread of a warp
__device__ __forceinline__ void wait1(const Ctl& c, uint32_t bar, uint32_t parity) {
    if (!mbar_try(bar, parity)) wait_slow(c, bar, parity);
}
// a whole warp
__device__ __forceinline__ void wait(const Ctl& c, uint32_t bar, uint32_t parity) {
    wait1(c, bar, parity);
    __syncwarp();
}

// The pieces of a block's share, walked alike by all of its warps.
struct Walk {
    long long x, end, W;
    int ncta, n_items, units_shared;
    const AttnItem* items;
};
__device__ __forceinline__ Walk walk_begin(const AttnParams& p, int cta) {
    const AttnHead* h = attn_head(p);
    Walk w;
    w.W = h->W;
    w.ncta = h->ncta;
    w.units_shared = h->units_shared;
    w.items = ws_ptr<AttnItem>(p.ws, p.L.item);
    w.n_items = p.G + p.S;
    w.x = w.end = 0;
    if (cta < w.ncta) {
        w.x = attn_cut(w.W, w.ncta, cta);
        w.end = attn_cut(w.W, w.ncta, cta + 1);
    }
    return w;
}
__device__ __forceinline__ bool walk_next(const AttnParams& p, Walk& w, int cta, AttnItem& it, AttnPiece& c) {
    if (w.x >= w.end) return false;
    const int ii = attn_find(w.items, w.n_items, w.x);
    it = w.items[ii];
    long long next;
    c = attn_piece(p, it, ii >= p.G, w.x, w.end, cta, w.units_shared, next);
    w.x = next;
    return true;
}

// ---- producer ----

template <int D>
__device__ void tc_producer(const AttnParams& p, const CUtensorMap* mk, const CUtensorMap* mv, const Ctl& ctl,
                            TcShared* sh, uint32_t ring, int lane) {
    using G = TcGeo<D>;
    const int box = p.page_size < kTile ? p.page_size : kTile;  // rows of one copy
    const int nbox = kTile / box;
    const int b = lane % nbox, half = lane / nbox;
    const bool on = half < G::kHalves;
    const uint32_t to = half * kHalf + b * box * 128;
    Walk w = walk_begin(p, blockIdx.x);
    AttnItem it;
    AttnPiece c;
    uint32_t f = 0;
    while (walk_next(p, w, blockIdx.x, it, c)) {
        const int keys = c.own ? __ldg(p.ctx_len + c.seq) + it.nodes : INT_MAX;
        const int32_t* row = p.table + (long long)c.seq * p.pages_per_seq;
        auto page_of = [&](int t) {
            const int pos = t * kTile + b * box;
            return t < c.t1 && pos < keys ? __ldg(row + (pos >> p.page_shift)) : -1;
        };
        int id = page_of(c.t0);
        for (int t = c.t0; t < c.t1; ++t) {
            const int next_id = page_of(t + 1);
            const int pos = t * kTile + b * box;
            const int boxes = min(nbox, (int)(((long long)keys - t * kTile + box - 1) / box));
            if (pos < keys && (id < 0 || id >= p.num_pages)) {
                raise_error(p.ws, kErrRange);
                id = 0;
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++f) {
                const uint32_t st = f % G::kStages, n = f / G::kStages;
                if (n > 0) wait(ctl, smem_u32(&sh->empty[st]), (n - 1) & 1);
                if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(ctl.abort))) return;
                const uint32_t bar = smem_u32(&sh->full[st]);
                if (lane == 0) mbar_expect_tx(bar, (uint32_t)(boxes * box * 128 * G::kHalves));
                __syncwarp();
                if (on && b < boxes)
                    tma_tile(ring + st * G::kStage + to, kv ? mv : mk, half * 64, c.hkv * p.page_size + (pos & (p.page_size - 1)), id, bar);
            }
            id = next_id;
        }
    }
}

// ---- products ----

template <int D>
__device__ void tc_issue(const AttnParams& p, const Ctl& ctl, TcShared* sh, uint32_t sq, uint32_t ring, uint32_t tmem) {
    using G = TcGeo<D>;
    constexpr uint32_t is = instruction(kTile, 0), io = instruction(D, 1);
    Walk w = walk_begin(p, blockIdx.x);
    AttnItem it;
    AttnPiece c;
    uint32_t f0 = 0, pieces = 0, np[2] = {0, 0};
    while (walk_next(p, w, blockIdx.x, it, c)) {
        const int n = c.t1 - c.t0;
        const bool two = c.rows > kTile;
        wait1(ctl, smem_u32(&sh->q_full), pieces & 1);
        ++pieces;
        tc_fence_after();
        const int steps = two ? n : (n + 1) / 2;
        for (int i = 0; i <= steps; ++i) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                // tile of this stream's previous and present step
                const int tp = two ? i - 1 : 2 * (i - 1) + s, tn = two ? i : 2 * i + s;
                if (i > 0 && tp < n) {
                    const uint32_t f = f0 + 2 * tp + 1, st = f % G::kStages;
                    wait1(ctl, smem_u32(&sh->full[st]), (f / G::kStages) & 1);
                    wait1(ctl, smem_u32(&sh->p_full[s]), np[s] & 1);
                    ++np[s];
                    tc_fence_after();
                    const uint64_t vb = operand(ring + st * G::kStage);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ts(tmem + 256 + 128 * s, tmem + 128 * s + 8 * k, vb + (uint64_t)((k * 2048) >> 4), io, i > 1 || k > 0);
                    if (!two || s == 1) tc_commit(smem_u32(&sh->empty[st]));
                    tc_commit(smem_u32(&sh->o_full[s]));
                }
                if (i < steps && tn < n) {
                    const uint32_t f = f0 + 2 * tn, st = f % G::kStages;
                    wait1(ctl, smem_u32(&sh->full[st]), (f / G::kStages) & 1);
                    tc_fence_after();
                    const uint64_t qa = operand(sq + (two ? s * G::kStage : 0)), kb = operand(ring + st * G::kStage);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t at = (uint64_t)(((k / 4) * kHalf + (k % 4) * 32) >> 4);
                        mma_ss(tmem + 128 * s, qa + at, kb + at, is, k > 0);
                    }
                    if (!two || s == 1) tc_commit(smem_u32(&sh->empty[st]));
                    tc_commit(smem_u32(&sh->s_full[s]));
                }
            }
        }
        f0 += 2 * n;
    }
}

// ---- rows ----

// Zeroes what the product with V must not meet in one key's row of one half: everything past the end,
// NaN and infinities in nodes (rows of zero weight would turn them into NaN). True if there were some.
__device__ __forceinline__ bool clean_row(uint32_t half, int k, bool past) {
    bool found = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t at = half + k * 128 + i * 16;
        uint32_t v[4];
        if (past) {
            v[0] = v[1] = v[2] = v[3] = 0;
        } else {
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u, bad = true;
                if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0x0000ffffu, bad = true;
            }
            if (!bad) continue;
            found = true;
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    }
    return found;
}

// Which of 32 positions from `base` on a row sees.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
__device__ __forceinline__ uint32_t seen32(const AttnParams& p, const uint32_t* mask_row, int node, int ctx, int keys, int base) {
    const int j0 = base - ctx;
    uint32_t nodes;
    if (mask_row) {
        const int wd = j0 >> 5, sh = j0 & 31;  // floor
        const uint32_t lo = wd >= 0 && wd < p.words ? __ldg(mask_row + wd) : 0u;
        const uint32_t hi = wd + 1 >= 0 && wd + 1 < p.words ? __ldg(mask_row + wd + 1) : 0u;
        nodes = __funnelshift_r(lo, hi, sh);
    } else {
        nodes = low_bits(node + 1 - j0);
    }
    return (low_bits(-j0) | nodes) & low_bits(keys - base);
}

template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, const AttnPiece& c, size_t orow, int rr, int col, const float* v, float inv) {
    if (c.whole) {
        uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + col);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            to[i] = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                               pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
    } else {
        float4* to = reinterpret_cast<float4*>(c.o + (size_t)rr * D + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

// NaN and infinities that were kept out of the product: added to the 32 columns just stored where the row
// sees their node (an infinity over the sum, or times a later factor, is the same infinity).
template <int D>
__device__ __forceinline__ void add_poison(const AttnParams& p, const AttnPiece& c, int nodes, const uint32_t* mask_row, int node, int ctx,
                                        size_t orow, int rr, int col) {
    const int j0 = max(0, c.t0 * kTile - ctx), j1 = min(nodes, c.t1 * kTile - ctx);
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        const bool sees = mask_row ? (__ldg(mask_row + (j >> 5)) >> (j & 31)) & 1u : j <= node;
        if (!sees) continue;
        const int pos = ctx + j;
        const size_t page = attn_page(p, c.seq, pos >> p.page_shift);
        const uint16_t* from =
            static_cast<const uint16_t*>(p.v_cache) + ((page * p.Hkv + c.hkv) * p.page_size + (pos & (p.page_size - 1))) * D + col;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            const uint32_t b = __ldg(from + i);
            if ((b & 0x7f80u) != 0x7f80u) continue;
            const float v = __uint_as_float(b << 16);
            if (c.whole) {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + orow * D + col + i;
                *to = __float2bfloat16_rn(__bfloat162float(*to) + v);
            } else {
                c.o[(size_t)rr * D + col + i] += v;
            }
        }
    }
}

template <int D>
__device__ void tc_rows(const AttnParams& p, const Ctl& ctl, TcShared* sh, unsigned char* sq, uint32_t ring, uint32_t tmem) {
    using G = TcGeo<D>;
    const int tid = threadIdx.x, lane = tid & 31, s = tid >> 7, r = tid & 127, quad = (tid >> 5) & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s;
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;  // a negative scale goes into q
    const float scale = fabsf(p.scale2) > 0.0f ? fabsf(p.scale2) : 1e-30f;  // 0: equal weights, and -inf stays -inf
    Walk w = walk_begin(p, blockIdx.x);
    AttnItem it;
    AttnPiece c;
    uint32_t f0 = 0, steps0[2] = {0, 0};  // fills and steps of earlier pieces
    while (walk_next(p, w, blockIdx.x, it, c)) {
        const int n = c.t1 - c.t0;
        const bool two = c.rows > kTile;
        const int ctx = c.own ? __ldg(p.ctx_len + c.seq) : INT_MAX, keys = c.own ? ctx + it.nodes : INT_MAX;
        // q: a block of 128 rows for each stream, or one for both
        const int rows_q = min(c.rows, 2 * kTile);
        for (int i = tid; i < rows_q * (D / 8); i += 256) {
            const int rr = i / (D / 8), ch = i - rr * (D / 8);
            const int row = c.row0 + rr, node = row / p.gq, hq = c.hkv * p.gq + (row - node * p.gq);
            uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                           (size_t)(c.node0 + node) * p.q_stride + (size_t)hq * D + ch * 8));
            v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
            const int k = rr & (kTile - 1);
            *reinterpret_cast<uint4*>(sq + (rr / kTile) * G::kStage + (ch / 8) * kHalf + k * 128 + (((ch & 7) ^ (k & 7)) << 4)) = v;
        }
        if (tid == 0) sh->poison = 0;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->q_full));
        rows_sync();  // poison is clear
        const int rr = two ? s * kTile + r : r;  // row of the unit's block
        const bool active = quad * 32 + (two ? s * kTile : 0) < c.rows;
        const bool mine = rr < c.rows;
        const int row = c.row0 + (mine ? rr : 0), node = row / p.gq, hq = c.hkv * p.gq + (row - node * p.gq);
        const uint32_t* mask_row = p.mask ? p.mask + (long long)(c.node0 + node) * p.words : nullptr;
        const int steps = two ? n : (n + 1 - s) / 2;  // tiles of this stream
        float m = kNegInf, l = 0.0f;                  // reference (times scale), sum
        for (int i = 0; i < steps; ++i) {
            const int tt = two ? i : 2 * i + s, pos0 = (c.t0 + tt) * kTile;
            const uint32_t step = steps0[s] + i;
            const bool tail = c.own && pos0 + kTile > ctx;
            if (tail) {
                const uint32_t f = f0 + 2 * tt + 1, st = f % G::kStages;
                wait(ctl, smem_u32(&sh->full[st]), (f / G::kStages) & 1);
                const uint32_t v = ring + st * G::kStage;
                bool found = false;
                const int k = two ? tid >> 1 : r;
                if (pos0 + k >= ctx) {
#pragma unroll
                    for (int h = 0; h < G::kHalves; ++h)
                        if (!two || G::kHalves == 1 || h == (tid & 1)) found |= clean_row(v + h * kHalf, k, pos0 + k >= keys);
                }
                if (found) sh->poison = 1;
                fence_async_smem();
                if (two) rows_sync();  // the other stream's product reads the same values
            }
            wait(ctl, smem_u32(&sh->s_full[s]), step & 1);
            if (active) {
                tc_fence_after();
                float z[kTile];
#pragma unroll
                for (int q = 0; q < 4; ++q) ld32(t_s + 32 * q, z + 32 * q);
                tc_wait_ld();
                if (tail) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t seen = seen32(p, mask_row, node, ctx, keys, pos0 + 32 * q);
#pragma unroll
                        for (int e = 0; e < 32; ++e) z[32 * q + e] = (seen >> e) & 1u ? z[32 * q + e] : kNegInf;
                    }
                }
                float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int e = 0; e < kTile; e += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[q]) : "f"(z[e + 2 * q]), "f"(z[e + 2 * q + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                const bool grow = mine && (top > m + 8.0f || m == kNegInf);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? fmaxf(top, m) : m;
                    const float fac = m == kNegInf ? 0.0f : (grow ? ex2(m - to) : 1.0f);
                    if (i > 0) {
                        wait(ctl, smem_u32(&sh->o_full[s]), (step - 1) & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            float o[32];
                            ld32(tmem + lanes + 256 + 128 * s + 32 * q, o);
                            tc_wait_ld();
                            uint32_t u[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * fac);
                            st32(tmem + lanes + 256 + 128 * s + 32 * q, u);
                        }
                        l *= fac;
                    }
                    m = to;
                }
                const float base = m == kNegInf ? 0.0f : -m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float a = ex2(fmaf(z[64 * q + 2 * e], scale, base)), b = ex2(fmaf(z[64 * q + 2 * e + 1], scale, base));
                        sum[(2 * e) & 3] += a;
                        sum[(2 * e + 1) & 3] += b;
                        pk[e] = pack_bf16(a, b);
                    }
                    st32(t_s + 32 * q, pk);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[s]));
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[s]));
            }
        }
        // the last products of the streams whose sums this thread reads
        const int steps_a = two ? n : (n + 1) / 2, steps_b = two ? n : n / 2;
        if (!two || s == 0) wait(ctl, smem_u32(&sh->o_full[0]), (steps0[0] + steps_a - 1) & 1);
        if ((!two && steps_b > 0) || (two && s == 1)) wait(ctl, smem_u32(&sh->o_full[1]), (steps0[1] + steps_b - 1) & 1);
        // with one block of rows the streams exchange their statistics where a second block of q would be
        float2* ml = reinterpret_cast<float2*>(sq + G::kStage);
        if (!two) ml[s * kTile + r] = make_float2(m, l);
        rows_sync();
        tc_fence_after();
        const bool poison = sh->poison != 0;
        if (quad * 32 + (two ? s * kTile : 0) < c.rows) {
            const size_t orow = (size_t)(c.node0 + node) * p.Hq + hq;
            float fa = 1.0f, fb = 0.0f;
            const bool join = !two && steps_b > 0;
            if (!two) {
                const float2 a = ml[r], b = ml[kTile + r];
                m = fmaxf(a.x, b.x);
                const float base = m == kNegInf ? 0.0f : m;
                fa = ex2(a.x - base);
                fb = ex2(b.x - base);
                l = a.y * fa + b.y * fb;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            // with one block of rows each group takes half of the columns
            const int c0 = two ? 0 : s * (D / 2), c1 = two ? D : c0 + D / 2;
#pragma unroll 1
            for (int col = c0; col < c1; col += 32) {
                float a[32], b[32];
                ld32(tmem + lanes + 256 + (two ? 128 * s : 0) + col, a);
                if (join) ld32(tmem + lanes + 384 + col, b);
                tc_wait_ld();
                if (join) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) a[e] = fmaf(a[e], fa, b[e] * fb);
                }
                if (mine) {
                    store_row<D>(p, c, orow, rr, col, a, inv);
                    if (poison) add_poison<D>(p, c, it.nodes, mask_row, node, ctx, orow, rr, col);
                }
            }
            if (mine && (two || s == 0)) {
                if (c.whole) {
                    if (p.lse) p.lse[orow] = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718056f;
                } else {
                    c.ml[rr] = make_float2(m, l);
                }
            }
        }
        tc_fence_before();
        rows_sync();  // sums and statistics have been read: the next piece may write over them
        f0 += 2 * n;
        steps0[0] += steps_a;
        steps0[1] += steps_b;
    }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using G = TcGeo<D>;
    extern __shared__ unsigned char dyn[];
    __shared__ TcShared shared;
    TcShared* sh = &shared;
    unsigned char* base = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    unsigned char* sq = base;
    const uint32_t ring = smem_u32(base + 2 * G::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(smem_u32(&sh->full[i]), 1);
            mbar_init(smem_u32(&sh->empty[i]), 1);
        }
        mbar_init(smem_u32(&sh->q_full), 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh->s_full[s]), 1);
            mbar_init(smem_u32(&sh->p_full[s]), 4);
            mbar_init(smem_u32(&sh->o_full[s]), 1);
        }
        sh->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const Ctl ctl{p.ws, &sh->abort};
    griddep_wait();
    griddep_launch_dependents();
    // 384 threads start with 168 registers each; the rows' eight warps go on with 216 and the other four
    // with 72 (2 x 216 + 72 = 3 x 168)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        tc_rows<D>(p, ctl, sh, sq, ring, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            tc_producer<D>(p, &mk, &mv, ctl, sh, ring, lane);
        } else if (warp == 9) {
            if (lane == 0) tc_issue<D>(p, ctl, sh, smem_u32(sq), ring, tmem);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*reinterpret_cast<volatile int*>(&sh->abort)) {
        // after a wait that ran out: give copies and products in flight time to land before the block's
        // shared and tensor memory is handed on
        const unsigned long long t0 = now_ns();
        while (now_ns() - t0 < 20000000ull) __nanosleep(1000);
    }
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A cache as [num_pages][Hkv * page_size][D], in boxes of 64 columns and up to 128 positions of one head.
bool encode_cache(CUtensorMap* m, const void* base, const AttnParams& p) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv * p.page_size, (cuuint64_t)p.num_pages};
    const cuuint64_t stride[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.D * 2 * p.Hkv * p.page_size};
    const cuuint32_t box[3] = {64, (cuuint32_t)(p.page_size < kTile ? p.page_size : kTile), 1}, one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc_t(const AttnParams& p, cudaStream_t st) {
    CUtensorMap mk, mv;
    if (!encode_cache(&mk, p.k_cache, p) || !encode_cache(&mv, p.v_cache, p)) return cudaErrorInvalidValue;
    auto kern = attn_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcGeo<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ncta_max);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = TcGeo<D>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, mk, mv);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnParams& p, cudaStream_t st) {
    return p.D == 64 ? launch_tc_t<64>(p, st) : launch_tc_t<128>(p, st);
}

}  // namespace smcsd
