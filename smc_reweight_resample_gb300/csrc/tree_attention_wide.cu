// tree_attention_wide.cu -- attention of drafted tokens over a paged bf16 cache on the tensor cores, for
// sequences with more than 128 rows.
//
// A row is a node and one of the query heads that share a key/value head. One block per SM walks its
// share of the line of key tiles (attn_plan.cuh); a tile is 128 keys.
//   warp 8     walks along the block's share, hands the pieces round and brings the pages of keys (attn_tc.cuh)
//   warp 10    brings the pages of values
//   warp 9     issues the products: S = Q K^T (128 rows x 128 keys, sums in tensor memory) and
//              O += P V with P read from tensor memory
//   (warp 11 idle: registers are handed over by fours)
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
#include "attn_tc.cuh"

namespace smcsd {

namespace {

constexpr int kTcThreads = 384;

template <int D>
struct TcGeo {
    static constexpr int kStage = TileGeo<D>::kBytes;  // one tile of keys or of values
    static constexpr int kKeys = D == 128 ? 2 : 5, kValues = D == 128 ? 3 : 5;  // stages
    static constexpr int kSmem = 1024 + 2 * kStage + (kKeys + kValues) * kStage;  // alignment, two blocks of q, the rings
};

template <int D>
struct __align__(8) TcShared {
    Ring<TcGeo<D>::kKeys> rk;
    Ring<TcGeo<D>::kValues> rv;
    PieceRing pieces;
    uint64_t q_full[2];  // by the piece's parity
    uint64_t s_full[2], p_full[2], o_full[2];
    uint32_t tmem;
    int abort;
    int poison;  // a NaN or infinity among the values of the piece's nodes
};

// ---- pieces, keys and values ----

// Two warps in one piece of code: the one with `keys` walks and brings the pages of keys, the other the pages of values.
template <int D, bool kPlanned>
__device__ void wide_fill(const AttnParams& p, bool keys, const CUtensorMap* map, const Ctl& ctl, TcShared<D>* sh, uint32_t ring, int lane) {
    using G = TcGeo<D>;
    Filler<D> filler(map, keys ? sh->rk.full : sh->rv.full, keys ? sh->rk.empty : sh->rv.empty, keys ? G::kKeys : G::kValues, ring);
    Walker<kPlanned> walk;
    if (keys) walk.begin(p, lane);
    int id = 0;
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        // the next piece, and its first ids, are fetched before this one's tiles have to wait for places
        int rows;
        if (keys) {
            PieceInfo next;
            walk.next(p, next, lane);
            sh->pieces.put(ctl, i, next, lane);
            rows = next.rows;
        } else {
            rows = sh->pieces.get(ctl, i);
        }
        const int id_ahead = rows > 0 ? filler.page_id(p, sh->pieces.at(i), 0, lane) : 0;
        if (i > 0) {
            if (!filler.fill(p, ctl, sh->pieces.at(i - 1), id, lane)) return;
            if (!keys) sh->pieces.done(i - 1);
        }
        if (rows == 0) return;
        id = id_ahead;
    }
}

// ---- products ----

template <int D>
__device__ void tc_issue(const AttnParams& p, const Ctl& ctl, TcShared<D>* sh, uint32_t sq, uint32_t ring_k, uint32_t ring_v, uint32_t tmem) {
    using G = TcGeo<D>;
    constexpr uint32_t is = instruction(kTile, 0, 0), io = instruction(D, 0, 1);
    uint32_t f0 = 0, np[2] = {0, 0};
    for (uint32_t piece = 0;; ++piece) {
        const int rows = sh->pieces.get(ctl, piece);
        if (rows == 0) return;
        const int n = uniform(sh->pieces.at(piece).n), keys = uniform(sh->pieces.at(piece).end - sh->pieces.at(piece).key0);
        sh->pieces.done(piece);
        const bool two = rows > kTile;
        wait(ctl, smem_u32(&sh->q_full[piece & 1]), (piece >> 1) & 1);
        tc_fence_after();
        const int steps = two ? n : (n + 1) / 2;
#pragma unroll 1
        for (int i = 0; i <= steps; ++i) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                // tile of this stream's previous and present step
                const int tp = two ? i - 1 : 2 * (i - 1) + s, tn = two ? i : 2 * i + s;
                if (i > 0 && tp < n) {
                    const uint32_t f = f0 + tp, st = f % G::kValues;
                    wait(ctl, smem_u32(&sh->rv.full[st]), (f / G::kValues) & 1);
                    wait(ctl, smem_u32(&sh->p_full[s]), np[s] & 1);
                    ++np[s];
                    tc_fence_after();
                    const uint64_t vb = operand(ring_v + st * G::kStage, TileGeo<D>::kGroup, 1024);
                    const uint32_t more = i > 1;
                    const int steps_v = tile_steps(keys - tp * kTile);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            if (k < steps_v) mma_ts(tmem + 256 + 128 * s, tmem + 128 * s + 8 * k, vb + (uint64_t)((k * 2 * TileGeo<D>::kGroup) >> 4), io, k > 0 ? 1u : more);
                        if (!two || s == 1) tc_commit(smem_u32(&sh->rv.empty[st]));
                        tc_commit(smem_u32(&sh->o_full[s]));
                    }
                    __syncwarp();
                }
                if (i < steps && tn < n) {
                    const uint32_t f = f0 + tn, st = f % G::kKeys;
                    wait(ctl, smem_u32(&sh->rk.full[st]), (f / G::kKeys) & 1);
                    tc_fence_after();
                    const uint64_t qa = operand(sq + (two ? s * G::kStage : 0), TileGeo<D>::kGroup, 0),
                                   kb = operand(ring_k + st * G::kStage, TileGeo<D>::kGroup, 0);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t at = (uint64_t)(TileGeo<D>::step(k) >> 4);
                            mma_ss(tmem + 128 * s, qa + at, kb + at, is, k > 0);
                        }
                        if (!two || s == 1) tc_commit(smem_u32(&sh->rk.empty[st]));
                        tc_commit(smem_u32(&sh->s_full[s]));
                    }
                    __syncwarp();
                }
            }
        }
        f0 += n;
    }
}

// ---- rows ----

template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, const PieceInfo& c, size_t orow, int rr, int col, const float* v, float inv) {
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

// NaN and infinities that were kept out of the product: added to the columns just stored where the row
// sees their node (an infinity over the sum, or times a later factor, is the same infinity).
template <int D>
__device__ __forceinline__ void add_poison(const AttnParams& p, const PieceInfo& c, const uint32_t* mask_row, int node, size_t orow, int rr, int c0, int c1) {
    const int j0 = max(0, c.key0 - c.ctx), j1 = min(c.end, c.key0 + c.n * kTile) - c.ctx;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        const bool sees = mask_row ? (__ldg(mask_row + (j >> 5)) >> (j & 31)) & 1u : j <= node;
        if (!sees) continue;
        const int pos = c.ctx + j;
        const size_t page = attn_page(p, c.seq, pos >> p.page_shift);
        const uint16_t* from =
            static_cast<const uint16_t*>(p.v_cache) + ((page * p.Hkv + c.hkv) * p.page_size + (pos & (p.page_size - 1))) * D;
#pragma unroll 1
        for (int i = c0; i < c1; ++i) {
            const uint32_t b = __ldg(from + i);
            if ((b & 0x7f80u) != 0x7f80u) continue;
            const float v = __uint_as_float(b << 16);
            if (c.whole) {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + orow * D + i;
                *to = __float2bfloat16_rn(__bfloat162float(*to) + v);
            } else {
                c.o[(size_t)rr * D + i] += v;
            }
        }
    }
}

template <int D, bool kPlanned>
__device__ void tc_rows(const AttnParams& p, const Ctl& ctl, TcShared<D>* sh, unsigned char* sq, uint32_t ring_v, uint32_t tmem) {
    using G = TcGeo<D>;
    const int tid = threadIdx.x, lane = tid & 31, s = tid >> 7, r = tid & 127, quad = (tid >> 5) & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s;
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;  // a negative scale goes into q
    const float scale = fabsf(p.scale2) > 0.0f ? fabsf(p.scale2) : 1e-30f;  // 0: equal weights, and -inf stays -inf
    uint32_t f0 = 0, steps0[2] = {0, 0};  // fills and steps of earlier pieces
    int pending = 0;
    for (uint32_t piece = 0;; ++piece) {
        const int rows = sh->pieces.get(ctl, piece);
        if (rows_any<256>(rows == 0)) break;  // all eight warps or none: they meet at barriers below
        const PieceInfo& c = sh->pieces.at(piece);
        const int n = c.n, first_tail = c.first_tail(7);
        const bool two = rows > kTile;
        // q: a block of 128 rows for each stream, or one for both
        const int rows_q = min(rows, 2 * kTile);
#pragma unroll 2
        for (int i = tid; i < rows_q * (D / 8); i += 256) {
            const int rr = i / (D / 8), ch = i - rr * (D / 8);
            const int row = c.row0 + rr, node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
            uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                           (size_t)(c.node0 + node) * p.q_stride + (size_t)hq * D + ch * 8));
            v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
            const int k = rr & (kTile - 1);
            *reinterpret_cast<uint4*>(sq + (rr / kTile) * G::kStage + TileGeo<D>::at(k, ch)) = v;
        }
        if (tid == 0) sh->poison = 0;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->q_full[piece & 1]));
        rows_sync<256>();  // poison is clear
        const int rr = two ? s * kTile + r : r;  // row of the unit's block
        const bool active = quad * 32 + (two ? s * kTile : 0) < rows;
        const bool mine = rr < rows;
        const int row = c.row0 + (mine ? rr : 0), node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
        const uint32_t* mask_row = p.mask ? p.mask + (long long)(c.node0 + node) * p.words : nullptr;
        const int steps = two ? n : (n + 1 - s) / 2;  // tiles of this stream
        float m = kNegInf, l = 0.0f;                  // reference (times scale), sum
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            const int tt = two ? i : 2 * i + s;
            const uint32_t step = steps0[s] + i;
            const bool tail = tt >= first_tail;
            wait(ctl, smem_u32(&sh->s_full[s]), step & 1);
            if (tail) {
                // The scores are there, and with them the products with the values of two tiles before: the
                // stage's earlier fill has landed, so this one may be waited for.
                const uint32_t f = f0 + tt, st = f % G::kValues;
                wait(ctl, smem_u32(&sh->rv.full[st]), (f / G::kValues) & 1);
                const int pos0 = c.key0 + tt * kTile;
                // by both groups where both have the tile
                if (clean_values<D>(ring_v + st * G::kStage, max(c.ctx - pos0, 0), c.end - pos0, two ? tid : r, two ? 256 : 128)) sh->poison = 1;
                fence_async_smem();
                if (two) rows_sync<256>();  // the other stream's product reads the same values
            }
            if (active) {
                tc_fence_after();
                float z[kTile];
#pragma unroll
                for (int q = 0; q < 4; ++q) ld32(t_s + 32 * q, z + 32 * q);
                tc_wait_ld();
                if (tail) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t seen = seen32(p, mask_row, node, c.ctx, c.end, c.key0 + tt * kTile + 32 * q);
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
        // the stream's last product; the other's is known to be done behind the next barrier
        const int steps_a = two ? n : (n + 1) / 2, steps_b = two ? n : n / 2;
        if (steps > 0) wait(ctl, smem_u32(&sh->o_full[s]), (steps0[s] + steps - 1) & 1);
        // with one block of rows the streams exchange their statistics where a second block of q would be
        float2* ml = reinterpret_cast<float2*>(sq + G::kStage);
        if (!two) ml[s * kTile + r] = make_float2(m, l);
        rows_sync<256>();
        tc_fence_after();
        const bool poison = sh->poison != 0;
        if (quad * 32 + (two ? s * kTile : 0) < rows) {
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
                if (mine) store_row<D>(p, c, orow, rr, col, a, inv);
            }
            if (mine && poison) add_poison<D>(p, c, mask_row, node, orow, rr, c0, c1);
            if (mine && (two || s == 0)) {
                if (c.whole) {
                    if (p.lse) p.lse[orow] = attn_lse(m, l);
                } else {
                    c.ml[rr] = make_float2(m, l);
                }
            }
        }
        tc_fence_before();
        rows_sync<256>();  // sums and statistics have been read: the next piece may write over them
        f0 += n;
        steps0[0] += steps_a;
        steps0[1] += steps_b;
        if (!kPlanned && c.join > 0) {
            if (tid == 0) sh->pieces.pending[pending] = c;
            ++pending;
        }
        sh->pieces.done(piece);
    }
    if (!kPlanned && pending > 0)  // behind the barrier of the loop's end
        attn_join_last<1, D, 8, 2>(p, sh->pieces.pending, pending, tid, 256, sh->pieces.last, [] { rows_sync<256>(); });
}

template <int D, bool kPlanned>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using G = TcGeo<D>;
    extern __shared__ unsigned char dyn[];
    __shared__ TcShared<D> shared;
    TcShared<D>* sh = &shared;
    unsigned char* base = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    unsigned char* sq = base;
    const uint32_t ring_k = smem_u32(base + 2 * G::kStage), ring_v = ring_k + G::kKeys * G::kStage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh->rk.init();
        sh->rv.init();
        sh->pieces.init(10);
        mbar_init(smem_u32(&sh->q_full[0]), 8);
        mbar_init(smem_u32(&sh->q_full[1]), 8);
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
        tc_rows<D, kPlanned>(p, ctl, sh, sq, ring_v, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 9)
            tc_issue<D>(p, ctl, sh, smem_u32(sq), ring_k, ring_v, tmem);
        else if (warp != 11)
            wide_fill<D, kPlanned>(p, warp == 8, warp == 8 ? &mk : &mv, ctl, sh, warp == 8 ? ring_k : ring_v, lane);
    }
    tc_fence_before();
    __syncthreads();
    settle(ctl);
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

template <int D>
static cudaError_t launch_wide_t(const AttnParams& p, cudaStream_t st) {
    return launch_tc(p.planned ? attn_wide_kernel<D, true> : attn_wide_kernel<D, false>, kTcThreads, TcGeo<D>::kSmem, p, st);
}

cudaError_t launch_attn_wide(const AttnParams& p, cudaStream_t st) {
    return p.D == 64 ? launch_wide_t<64>(p, st) : launch_wide_t<128>(p, st);
}

}  // namespace smcsd
