// tree_attention_wide.cu -- attention of drafted tokens over a paged bf16 cache on the tensor cores, for
// sequences of many rows (the rule is kind_of's).
//
// A row is a node and one of the query heads that share a key/value head. One block per SM walks its
// share of the line of key tiles (attn_plan.cuh); a tile is 128 keys.
//   warps 0-7      two groups of four, one thread per row: maximum, exponentials, sum, and P (bf16) written
//                  over S in tensor memory
//   warp 8         walks along the block's share, hands the pieces round and brings the pages of keys (attn_tc.cuh)
//   warp 10        brings the pages of values
//   warps 9 and 11 issue one group's products each: S = Q K^T (128 rows x 128 keys, sums in tensor memory) and
//                  O += P V with P read from tensor memory
// The groups are two streams that take turns on the tensor core: while one does its exponentials the
// products of the other run. With more than 128 rows in a unit the streams are two blocks of 128 rows
// over the same tiles; with fewer they are the even and the odd tiles of the same rows, joined at the
// end. Tensor memory is full (twice 128 columns of S and of O), so P lies over S and a stream's next S follows its
// last product with V. The softmax goes through a tile in two halves of 64 keys: half the registers (none of the loop's
// values is spilled), and the first half's product runs during the second one's exponentials.
//
// 8 trees of up to 64 nodes over up to 32768 tokens, 64 query heads on 8, D = 128: 310 us, 0.88 PFLOP/s (45 % of the
// measured bf16 rate; 140 us). What bounds it is a stream's chain: of 4200 clocks for a tile a group computes 1700, waits 1600 for
// its next scores (last weights -> product -> scores -> commit) and spends the rest between; the products of both streams
// take 2200. Measured otherwise: one warp issuing for both streams 356 us, scores by halves of 64 keys in two buffers 408 us
// (a product of 64 keys takes as long as one of 128, since reading Q bounds it), and the last step of a piece by stores
// along the rows 330 us.
//
// Softmax. With z = scale2 q.k (in units of log 2), a row keeps a reference m, l = sum exp2(z - m) and
// O = sum exp2(z - m) V. The reference moves (and O is rescaled) only when the maximum has grown by more
// than 8, so weights stay below 2^8: sums are in float32, P has bf16's 8 bits at any scale. l sums the
// weights before they are rounded. P is rounded to bf16 because the two operands of a product have one type and V is bf16:
// each weight is off by up to 2^-8 of itself with either sign, about as much as the rounding of the result (values of either
// sign: 0.0015 of the result's norm, beside 0.0017 for its own rounding). More bits would take a V converted to 32 bits (twice
// the shared memory and half the rate), or P in two parts and twice the products, which bound this kernel.
#include "attn_tc.cuh"

namespace smcsd {

namespace {

constexpr int kTcThreads = 384;

template <int D>
struct TcGeo {
    static constexpr int kStage = TileGeo<D>::kBytes;  // one tile of keys or of values
    static constexpr int kKeys = D == 128 ? 2 : 5, kValues = D == 128 ? 3 : 5;  // stages
    // 2 KB of statistics: where a second block of q would be, or (the eight warps' 4 KB for outputs take two blocks of 64 columns)
    // behind the rings
    static constexpr int kStats = D == 128 ? kStage : (2 + kKeys + kValues) * kStage;
    static constexpr int kSmem = 1024 + (2 + kKeys + kValues) * kStage + (D == 128 ? 0 : 2048);  // alignment, two blocks of q, the rings
};

template <int D>
struct __align__(8) TcShared {
    Ring<TcGeo<D>::kKeys> rk;
    Ring<TcGeo<D>::kValues> rv;
    PieceRing pieces;
    uint64_t q_full[2];  // by the piece's parity
    uint64_t s_full[2], p_full[2][2], o_full[2][2];  // [stream][half of the tile]
    uint64_t v_clean[TcGeo<D>::kValues];  // [stage] the first stream's warp has cleaned the values for both
    uint32_t tmem;
    int abort;
    uint32_t poison[kPieces];  // i + 1: a NaN or infinity among the values of the i-th piece's nodes
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

// One warp for each stream. Its products follow one another: a tile's scores are written over the weights of its tile before,
// behind the product that reads them. Both warps watch all tiles land and report all of them as read, so that neither falls
// a round of the rings behind where the streams take turns on the tiles.
template <int D>
__device__ void wide_products(const AttnParams& p, const Ctl& ctl, TcShared<D>* sh, int s, uint32_t sq, uint32_t ring_k, uint32_t ring_v,
                              uint32_t tmem) {
    using G = TcGeo<D>;
    constexpr uint32_t is = instruction(kTile, 0, 0), io = instruction(D, 0, 1);
    const uint32_t t_s = tmem + 128 * s, t_o = tmem + 256 + 128 * s;
    uint32_t used = 0, tails = 0;  // parities of the weights and of the stages' cleaned values
    uint32_t kst = 0, kround = 0, vst = 0, vround = 0;
    for (uint32_t piece = 0;; ++piece) {
        const int rows = sh->pieces.get(ctl, piece);
        if (rows == 0) return;
        const PieceInfo& c = sh->pieces.at(piece);
        const int n = uniform(c.n), keys = uniform(c.end - c.key0), first_tail = c.first_tail(7);
        const bool two = rows > kTile;
        wait(ctl, smem_u32(&sh->q_full[piece & 1]), (piece >> 1) & 1);
        const uint64_t qa = operand(sq + (two ? s * G::kStage : 0), TileGeo<D>::kGroup, 0);
        int ts = 0, to = 0;  // tiles whose keys, whose values have landed
        // own: this stream's next tile whose scores are issued (n or more: none is left)
#pragma unroll 1
        for (int own = two ? 0 : s, before = -1;; before = own, own += two ? 1 : 2) {
            uint32_t v = 0, vbar = 0;
            int steps = 0;
            if (before >= 0) {
#pragma unroll 1
                for (; to <= before; ++to) {
                    wait(ctl, smem_u32(&sh->rv.full[vst]), vround & 1);
                    vbar = smem_u32(&sh->rv.empty[vst]);
                    v = ring_v + vst * G::kStage;
                    if (to < before) {
                        if (elect_one()) mbar_arrive(vbar);
                    } else if (to >= first_tail) {  // while the weights are worked out
                        if (!two || s == 0) {
                            if (clean_values<D>(v, max(c.ctx - c.key0 - to * kTile, 0), keys - to * kTile, threadIdx.x & 31, 32))
                                *reinterpret_cast<volatile uint32_t*>(&sh->poison[piece % kPieces]) = piece + 1;
                            fence_async_smem();
                            __syncwarp();
                            if (two && elect_one()) mbar_arrive(smem_u32(&sh->v_clean[vst]));
                        } else {
                            wait(ctl, smem_u32(&sh->v_clean[vst]), (tails >> vst) & 1);
                            tails ^= 1u << vst;
                            fence_async_smem();
                        }
                    }
                    __syncwarp();
                    if (++vst == G::kValues) vst = 0, ++vround;
                }
                steps = tile_steps(keys - before * kTile);
                const uint32_t more = before > (two ? 0 : s);
                const uint64_t vb = operand(v, TileGeo<D>::kGroup, 1024);
                wait(ctl, smem_u32(&sh->p_full[s][0]), used & 1);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps) mma_ts(t_o, t_s + 8 * k, vb + (uint64_t)((k * 2 * TileGeo<D>::kGroup) >> 4), io, k > 0 ? 1u : more);
                    tc_commit(smem_u32(&sh->o_full[s][0]));
                    mbar_arrive(smem_u32(&sh->o_full[s][0]));  // orders the piece's poison before it
                }
                __syncwarp();
            }
            // keys for the next scores, before the weights that they wait for
            uint32_t k0 = 0, kbar = 0;
#pragma unroll 1
            for (; ts < n && ts <= own; ++ts) {
                wait(ctl, smem_u32(&sh->rk.full[kst]), kround & 1);
                kbar = smem_u32(&sh->rk.empty[kst]);
                k0 = ring_k + kst * G::kStage;
                if (ts < own && elect_one()) mbar_arrive(kbar);
                __syncwarp();
                if (++kst == G::kKeys) kst = 0, ++kround;
            }
            const uint64_t kb = operand(k0, TileGeo<D>::kGroup, 0), vb = operand(v + 8 * TileGeo<D>::kGroup, TileGeo<D>::kGroup, 1024);
            if (before >= 0) wait(ctl, smem_u32(&sh->p_full[s][1]), used & 1);
            tc_fence_after();
            if (elect_one()) {
                if (before >= 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 + k < steps) mma_ts(t_o, t_s + 64 + 8 * k, vb + (uint64_t)((k * 2 * TileGeo<D>::kGroup) >> 4), io, 1u);
                    tc_commit(vbar);
                    tc_commit(smem_u32(&sh->o_full[s][1]));
                    mbar_arrive(smem_u32(&sh->o_full[s][1]));
                }
                if (own < n) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t at = (uint64_t)(TileGeo<D>::step(k) >> 4);
                        mma_ss(t_s, qa + at, kb + at, is, k > 0);
                    }
                    tc_commit(kbar);
                    tc_commit(smem_u32(&sh->s_full[s]));
                }
            }
            __syncwarp();
            if (before >= 0) ++used;
            if (own >= n) break;
        }
        // the other stream's last tile
#pragma unroll 1
        for (; to < n; ++to) {
            wait(ctl, smem_u32(&sh->rv.full[vst]), vround & 1);
            if (elect_one()) mbar_arrive(smem_u32(&sh->rv.empty[vst]));
            __syncwarp();
            if (++vst == G::kValues) vst = 0, ++vround;
        }
        sh->pieces.done(piece);
    }
}

// ---- rows ----

// 32 columns of a warp's 32 rows, a lane's row in v, to the result or the slot (`to`: the lane's row of the result). They pass
// through 4 KB of shared memory, after which eight lanes have a row's 128 bytes: stores by rows touched 32 lines each, and
// those of a piece of 256 rows took 8000 clocks.
template <int D>
__device__ __forceinline__ void store_rows(const AttnParams& p, const PieceInfo& c, unsigned char* stage, int row0, int count, int to, int col,
                                           const float* v, int lane) {
    float4* st = reinterpret_cast<float4*>(stage);
#pragma unroll
    for (int x = 0; x < 8; ++x) st[lane * 8 + (x ^ (lane & 7))] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
    __syncwarp();
    const bool whole = c.whole;
    float* o = c.o + (size_t)row0 * D + col;
#pragma unroll 4
    for (int x = 0; x < 8; ++x) {
        const int r = 4 * x + (lane >> 3), part = lane & 7;
        const float4 f = st[r * 8 + (part ^ (r & 7))];
        const int at = __shfl_sync(0xffffffffu, to, r);
        if (r >= count) continue;
        if (whole)
            attn_store4<1>(p.out, (size_t)at * D + col + 4 * part, f);
        else
            *reinterpret_cast<float4*>(o + r * D + 4 * part) = f;
    }
    __syncwarp();
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
__device__ void tc_rows(const AttnParams& p, const Ctl& ctl, TcShared<D>* sh, unsigned char* sq, uint32_t tmem) {
    using G = TcGeo<D>;
    const int tid = threadIdx.x, lane = tid & 31, s = tid >> 7, r = tid & 127, quad = (tid >> 5) & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s;
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;  // a negative scale goes into q
    const float scale = fabsf(p.scale2) > 0.0f ? fabsf(p.scale2) : 1e-30f;  // 0: equal weights, and -inf stays -inf
    uint32_t steps0[2] = {0, 0};  // steps of earlier pieces
    int pending = 0;
    for (uint32_t piece = 0;; ++piece) {
        const int rows = sh->pieces.get(ctl, piece);
        if (rows_any<256>(rows == 0)) break;  // all eight warps or none: they meet at barriers below
        const PieceInfo& c = sh->pieces.at(piece);
        const int n = c.n, first_tail = c.first_tail(7);
        const bool two = rows > kTile;
        // q: a block of 128 rows for each stream, or one for both
        const int rows_q = min(rows, 2 * kTile);
#pragma unroll 1
        for (int i0 = tid; i0 < rows_q * (D / 8); i0 += 8 * 256) {  // eight loads in flight
            uint4 v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int i = min(i0 + 256 * y, rows_q * (D / 8) - 1), rr = i / (D / 8), ch = i - rr * (D / 8);
                const int row = c.row0 + rr, node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
                v[y] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                            (size_t)(c.node0 + node) * p.q_stride + (size_t)hq * D + ch * 8));
            }
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int i = i0 + 256 * y, rr = i / (D / 8), ch = i - rr * (D / 8);
                if (rr >= rows_q) continue;
                v[y].x ^= flip, v[y].y ^= flip, v[y].z ^= flip, v[y].w ^= flip;
                *reinterpret_cast<uint4*>(sq + (rr / kTile) * G::kStage + TileGeo<D>::at(rr & (kTile - 1), ch)) = v[y];
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->q_full[piece & 1]));
        const int rr = two ? s * kTile + r : r;  // row of the unit's block
        const bool active = quad * 32 + (two ? s * kTile : 0) < rows;
        const bool mine = rr < rows;
        const int row = c.row0 + (mine ? rr : 0), node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
        const uint32_t* mask_row = p.mask ? p.mask + (long long)(c.node0 + node) * p.words : nullptr;
        const int steps = two ? n : (n + 1 - s) / 2;  // tiles of this stream
        float m = kNegInf, l = 0.0f;                  // reference (times scale), sum
#pragma unroll 1
        for (int x = 0; x < 2 * steps; ++x) {
            const int i = x >> 1, h = x & 1, tt = two ? i : 2 * i + s;
            const uint32_t step = steps0[s] + i;
            const bool tail = tt >= first_tail;
            if (h == 0) wait(ctl, smem_u32(&sh->s_full[s]), step & 1);
            if (active) {
                const uint32_t at_s = t_s + 64 * h;
                tc_fence_after();
                float z[64];
                ld32(at_s, z);
                ld32(at_s + 32, z + 32);
                tc_wait_ld();
                if (tail) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t seen = seen32(p, mask_row, node, c.ctx, c.end, c.key0 + tt * kTile + 64 * h + 32 * q);
#pragma unroll
                        for (int e = 0; e < 32; ++e) z[32 * q + e] = (seen >> e) & 1u ? z[32 * q + e] : kNegInf;
                    }
                }
                float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int e = 0; e < 64; e += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[q]) : "f"(z[e + 2 * q]), "f"(z[e + 2 * q + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                const bool grow = mine && (top > m + 8.0f || m == kNegInf);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? fmaxf(top, m) : m;
                    const float fac = m == kNegInf ? 0.0f : (grow ? ex2(m - to) : 1.0f);
                    if (x > 0) {
                        wait(ctl, smem_u32(&sh->o_full[s][h ^ 1]), (step - (h ^ 1)) & 1);  // the half before
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
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float a = ex2(fmaf(z[2 * e], scale, base)), b = ex2(fmaf(z[2 * e + 1], scale, base));
                    sum[(2 * e) & 3] += a;
                    sum[(2 * e + 1) & 3] += b;
                    pk[e] = pack_bf16(a, b);
                }
                st32(at_s, pk);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[s][h]));
        }
        // the stream's last product; the other's is known to be done behind the next barrier
        const int steps_a = two ? n : (n + 1) / 2, steps_b = two ? n : n / 2;
        if (steps > 0) wait(ctl, smem_u32(&sh->o_full[s][1]), (steps0[s] + steps - 1) & 1);
        // with one block of rows the streams exchange their statistics; the outputs pass through the place of the first block of q
        float2* ml = reinterpret_cast<float2*>(sq + G::kStats);
        if (!two) ml[s * kTile + r] = make_float2(m, l);
        rows_sync<256>();
        tc_fence_after();
        const bool poison = *reinterpret_cast<volatile uint32_t*>(&sh->poison[piece % kPieces]) == piece + 1;
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
                if (c.whole) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) a[e] *= inv;
                }
                const int row_w = quad * 32 + (two ? s * kTile : 0);  // this warp's first
                store_rows<D>(p, c, sq + (tid >> 5) * 4096, row_w, rows - row_w, (int)orow, col, a, lane);
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
        steps0[0] += steps_a;
        steps0[1] += steps_b;
        if (!kPlanned && c.join > 0) {
            if (tid == 0) sh->pieces.pending[pending] = c;
            ++pending;
        }
        sh->pieces.done(piece);
    }
    if (!kPlanned && pending > 0)  // behind the barrier of the loop's end
        attn_join_last<1, D, 8, 3>(p, sh->pieces.pending, pending, tid, 256, sh->pieces.last, [] { rows_sync<256>(); });
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
        sh->rk.init(2);
        sh->rv.init(2);
        sh->pieces.init(11);
        mbar_init(smem_u32(&sh->q_full[0]), 8);
        mbar_init(smem_u32(&sh->q_full[1]), 8);
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&sh->p_full[s >> 1][s & 1]), 4);
            mbar_init(smem_u32(&sh->o_full[s >> 1][s & 1]), 2);
        }
        mbar_init(smem_u32(&sh->s_full[0]), 1);
        mbar_init(smem_u32(&sh->s_full[1]), 1);
        for (int i = 0; i < G::kValues; ++i) mbar_init(smem_u32(&sh->v_clean[i]), 1);
        for (int i = 0; i < kPieces; ++i) sh->poison[i] = 0;
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
        tc_rows<D, kPlanned>(p, ctl, sh, sq, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 9 || warp == 11)
            wide_products<D>(p, ctl, sh, warp == 11, smem_u32(sq), ring_k, ring_v, tmem);
        else
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
