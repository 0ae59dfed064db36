// tree_attention_narrow.cu -- attention of drafted tokens over a paged bf16 cache on the tensor cores, for
// sequences of few rows (a row is a node and one of the query heads that share a key/value head; the rule is kind_of's).
//
// A unit of few rows is bound by the bytes of its keys and values, so the products are turned: the 128 keys of a
// tile are the rows of the tensor core's output and the query rows its columns,
//   S^T = K Q^T   (128 keys x N, in tensor memory),   O^T += V^T P^T   (D x N, in tensor memory),
// which costs N / 128 of the products of padded query rows, and a thread holds one key: 32 exponentials for
// each of 128 threads in place of 128 for each of 32. Blocks, tiles and cut are those of attn_plan.cuh.
//   warps 0-15  four groups of four, one thread per key and 32 columns: exponentials, sums, P (bf16) to shared
//               memory. With up to 32 rows the groups take four tiles at a time, with up to 64 two tiles in
//               two halves of the rows, above one tile in quarters: group w always has columns 32 w .. 32 w + 31
//               of the 128 that scores, weights and outputs have. A short piece of few rows is left to one group, so
//               that four of them are under way (Split).
//   warp 16     walks along the block's share, hands the pieces round in shared memory and brings the pages of keys
//               (attn_tc.cuh)
//   warp 18     brings the query rows (two places of 64 rows, or one of 128) and the pages of values
//   warps 17 and 19  issue S^T and O^T: one warp for both has more to issue than a tile's bytes take. Scores have two
//               buffers, so those of the next round of tiles are there when a group comes to them, and those of the next
//               piece while this one is written out. Warp 19 also cleans the values behind a tile's last key.
//
// Measured (D = 128 unless said): 64 chains of up to 21 nodes over up to 4096 tokens, 32 query heads on 8: 161 us, 5.1 TB/s
// (76 % of a copy's rate; 142 us with 8 nodes, where the wait for the four groups' barriers is shorter). 8 groups of
// 16 particles with 5 nodes over 2048 tokens, 90 % of them shared: 97 us with the planning and the joining kernel (8 and
// about 10): 1024 units of two tiles each, bound by the warps that fetch and issue, a few thousand clocks for each unit; the
// kernel's code (83 KB; 95 KB without a plan) does not stay in an SM's instruction cache, and what made it shorter, or took steps out of
// those warps' loops, made these units faster. 16 sequences with 5 nodes over 2048 tokens, 16 heads of 64: 34 us; one token
// over 517: 11.4 us, nearly all of it the first pass through the code and the chain of waits of one tile.
//
// Softmax. Per column: a reference m common to the keys of the group's tiles, P = exp2(z - m) with
// z = scale2 q.k, l the sum of P before it is rounded (each thread adds up its own keys; they meet at the end of
// the unit) and O. Any reference that keeps exp2 in range serves, so the maximum over the keys is not taken for
// each tile: a vote of the four warps asks whether some z - m is above 8, and only then (always in a group's first
// tile) the maximum of that column becomes the new reference and l and O are rescaled. Weights stay below 2^8;
// sums are in float32; P is rounded to bf16 for the product with V, as in the wide kernel.
#include "attn_tc.cuh"

namespace smcsd {

namespace {

constexpr int kTcThreads = 640, kSoftThreads = 512;
constexpr float kNone = -3.402823466e38f;  // reference of a column that has seen nothing: any score is above it

template <int D>
struct NarrowGeo {
    static constexpr int kStage = TileGeo<D>::kBytes;
    static constexpr int kKeys = D == 128 ? 2 : 5, kValues = D == 128 ? 3 : 6;  // stages
    static constexpr int kBlock = 128 * 128;     // 128 keys x 64 columns of P
    static constexpr int kWeights = 2 * kBlock;  // P: 128 columns x 128 keys
    static constexpr int kSlot = 8 * TileGeo<D>::kGroup;  // 64 query rows
    static constexpr int kSmem = 1024 + kStage + kWeights + (kKeys + kValues) * kStage;
};

template <int D>
struct __align__(16) NarrowShared {
    __align__(16) float m[kTile];  // references, read four at a time
    PieceRing pieces;
    Ring<NarrowGeo<D>::kKeys> rk;
    Ring<NarrowGeo<D>::kValues> rv;
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[4][2], o_full[4][2];  // [tile of a round, or a single group][buffer]
    uint64_t p_full[4][2];                // [group][buffer]
    uint32_t tmem;
    int abort;
    uint32_t poison[kPieces];  // i + 1: a NaN or infinity among the values of the i-th piece's nodes
};

// Places of the query rows: a piece of up to 64 rows takes the next of the two, a larger one both.
struct QuerySlots {
    uint32_t uses = 0;  // parities
    int next = 0, first, last;
    __device__ __forceinline__ void take(int rows) {
        const bool both = rows > 64;
        first = both ? 0 : next;
        last = both ? 2 : next + 1;
        next = both ? 0 : next ^ 1;
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) {  // f(place, parity of how often it was taken before)
#pragma unroll 1
        for (int x = first; x < last; ++x) f(x, (uses >> x) & 1u);
    }
    __device__ __forceinline__ void done() { uses ^= (1u << last) - (1u << first); }
};

// How a piece's rows and tiles are laid over the four groups: all of them on one piece, or (a short piece of few rows) the next
// group alone, so that up to four such pieces are under way and the waits of one are filled by the others. Short is up to 8
// tiles: 8 groups of 16 particles (two tiles in a unit) took 106.8 us with none, 101.4 / 99.2 / 99.5 / 99.1 with 1 / 2 / 4 / 8;
// 16 sequences of 17 tiles, cut between the blocks, 35.2 / 35.2 / 35.2 / 34.8 / 34.0.
constexpr int kSoloTiles = 8;
struct Split {
    int log_tiles;  // tiles of a round: 4, 2 or 1
    int log_chunks; // groups side by side on the rows of one tile: 1, 2 or 4
    int used;       // chunks that have rows
    bool solo;      // one group has it
    int first;      // that group, or the first one
    // `turn`: the group that takes the next such piece
    __device__ __forceinline__ Split(int rows, int n, int& turn) {
        solo = rows <= 32 && n <= kSoloTiles;
        log_chunks = (rows > 32) + (rows > 64);
        log_tiles = solo ? 0 : 2 - log_chunks;
        used = (rows + 31) >> 5;
        first = solo ? turn : 0;
        turn = (turn + solo) & 3;
    }
    // barriers and first group of tile k of a round
    __device__ __forceinline__ int bar(int k) const { return first + k; }
    __device__ __forceinline__ int group(int k) const { return first + (k << log_chunks); }
    __device__ __forceinline__ int tiles() const { return 1 << log_tiles; }
    __device__ __forceinline__ int chunks() const { return 1 << log_chunks; }
    // tiles of n that are number k of their round
    __device__ __forceinline__ int rounds(int n, int k) const { return (n - k + tiles() - 1) >> log_tiles; }
};

// How often the barriers of [k][buffer b] were used by earlier pieces: parities, bit 2 k + b.
struct Uses {
    uint32_t bits;
    __device__ __forceinline__ uint32_t parity(int k, int b, int use) const { return ((bits >> (2 * k + b)) ^ use) & 1u; }
    __device__ __forceinline__ void add(int n, const Split& sp) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int x = k - sp.first;
            const uint32_t r = x >= 0 && x < sp.tiles() ? sp.rounds(n, x) : 0;
            bits ^= (((r + 1) >> 1) & 1u) << (2 * k) | ((r >> 1) & 1u) << (2 * k + 1);
        }
    }
};

// ---- pieces, keys, query rows and values ----

// A piece's query rows, and rows of zeros (scores of zero) up to a multiple of 32. A lane has one 16-byte column and every
// second or fourth row: eight rows a turn, with a few additions each (a division for each row and a long address took 3000
// clocks for 32 rows, and this warp's turn for a piece was what bound short ones).
template <int D>
__device__ __forceinline__ void narrow_queries(const AttnParams& p, const PieceInfo& c, uint32_t to, int lane) {
    constexpr int kCols = D / 8, kStep = 32 / kCols;
    const int ch = lane % kCols, r0 = lane / kCols, node = attn_node(p, c.row0 + r0);
    int h = c.row0 + r0 - node * p.gq;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    const __nv_bfloat16* from = q + (size_t)(c.node0 + node) * p.q_stride + (size_t)(c.hkv * p.gq + h) * D + ch * 8;
    const int nodes = attn_node(p, kStep), heads = kStep - nodes * p.gq;  // from one row of this lane to the next
    const long long step = nodes * p.q_stride + heads * D, wrap = p.q_stride - (long long)p.gq * D;
    const uint32_t at = (uint32_t)((ch & 7) ^ r0) << 4;
    to += (ch >> 3) * 1024 + r0 * 128;
#pragma unroll 1
    for (int r = r0; r < ((c.rows + 31) & ~31); r += 8, to += TileGeo<D>::kGroup) {
#pragma unroll
        for (int y = 0; y < 8; y += kStep) {
            const bool there = r + y < c.rows;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + y * 128 + (at ^ (y << 4))), "l"(there ? from : q),
                         "r"(there ? 16 : 0)
                         : "memory");
            from += step;
            h += heads;
            if (h >= p.gq) h -= p.gq, from += wrap;
        }
    }
}

// Two warps in one piece of code (it is long): the one with `keys` walks and brings the pages of keys, the other the query rows
// and the pages of values. The next piece, its query rows and its first page ids are fetched before the present one's tiles have
// to wait for places.
template <int D, bool kPlanned>
__device__ void narrow_fill(const AttnParams& p, bool keys, const CUtensorMap* map, const Ctl& ctl, NarrowShared<D>* sh, uint32_t sq,
                            uint32_t ring, int lane) {
    using G = NarrowGeo<D>;
    Filler<D> filler(map, keys ? sh->rk.full : sh->rv.full, keys ? sh->rk.empty : sh->rv.empty, keys ? G::kKeys : G::kValues, ring);
    QuerySlots qs;
    Walker<kPlanned> walk;
    if (keys) walk.begin(p, lane);
    int id = 0, rows = 0;  // of the piece before
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        int rows_ahead;
        if (keys) {
            PieceInfo next;
            walk.next(p, next, lane);
            sh->pieces.put(ctl, i, next, lane);
            rows_ahead = next.rows;
        } else {
            rows_ahead = sh->pieces.get(ctl, i);
        }
        const PieceInfo &c = sh->pieces.at(i - 1), &ahead = sh->pieces.at(i);
        const bool more = rows_ahead > 0;
        const int id_ahead = more ? filler.page_id(p, ahead, 0, lane) : 0;
        // Query rows ahead of this piece's values only where they do not take its own places: those are free when its scores are
        // done, for which its values are needed.
        const bool early = max(rows, rows_ahead) <= 64;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            if (pass == 1 && i > 0 && !filler.fill(p, ctl, c, id, lane)) return;
            if (keys || !more || early != (pass == 0)) continue;
            qs.take(rows_ahead);
            qs.each([&](int x, uint32_t uses) { wait(ctl, smem_u32(&sh->q_empty[x]), uses ^ 1); });  // at once the first time
            narrow_queries<D>(p, ahead, sq + qs.first * G::kSlot, lane);
            // reported by the copies themselves; the warp that issues the scores has the fence
            qs.each([&](int x, uint32_t) {
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh->q_full[x])) : "memory");
            });
            __syncwarp();
            qs.done();
        }
        if (!keys && i > 0) sh->pieces.done(i - 1);
        if (!more) break;
        rows = rows_ahead;
        id = id_ahead;
    }
    // the last scores' reports land before the block ends
    if (!keys)
        for (int x = 0; x < 2; ++x) wait(ctl, smem_u32(&sh->q_empty[x]), ((qs.uses >> x) & 1) ^ 1);
}

// ---- products ----

// Parities of the groups' weights, as one issuing warp waits for them: bit 2 * group + buffer.
struct Weights {
    uint32_t bits = 0;
    template <int D>
    __device__ __forceinline__ void wait_for(const Ctl& ctl, NarrowShared<D>* sh, int bit) {
        wait(ctl, smem_u32(&sh->p_full[0][0]) + 8 * bit, (bits >> bit) & 1);
        bits ^= 1u << bit;
    }
};

// A buffer of scores is free when its group's weights are there (`out`: those not yet waited for). Where all groups take part in
// this piece or the one before, everybody has to be through with that one, since they wait for each other's barriers; pieces of
// single groups have barriers of their own.
template <int D>
__device__ void narrow_scores(const AttnParams& p, const Ctl& ctl, NarrowShared<D>* sh, uint32_t sq, uint32_t ring_k, uint32_t tmem) {
    using G = NarrowGeo<D>;
    Weights weights;
    QuerySlots qs;
    uint32_t st = 0, round = 0, out = 0;
    int turn = 0;
    bool solo = false;
    auto drain = [&](uint32_t some) {
        some &= out;
        out ^= some;
        for (; some; some &= some - 1) weights.wait_for(ctl, sh, __ffs(some) - 1);
    };
    for (uint32_t i = 0;; ++i) {
        const int rows = sh->pieces.get(ctl, i);
        if (rows == 0) return;
        const int n = uniform(sh->pieces.at(i).n);
        sh->pieces.done(i);
        const Split split(rows, n, turn);
        qs.take(rows);
        qs.each([&](int x, uint32_t uses) { wait(ctl, smem_u32(&sh->q_full[x]), uses); });
        fence_async_smem();
        if (!split.solo || !solo) drain(~0u);
        solo = split.solo;
        const uint32_t is = instruction(32 * split.used, 0, 0);
        const uint64_t qb = operand(sq + qs.first * G::kSlot, TileGeo<D>::kGroup, 0);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const int k = t & (split.tiles() - 1), b = (t >> split.log_tiles) & 1;
            // bits 2 * group + b of the tile's groups
            const uint32_t groups = ((1u << 2 * split.used) - 1) / 3 << (2 * split.group(k) + b);
            wait(ctl, smem_u32(&sh->rk.full[st]), round & 1);
            drain(groups);
            out |= groups;
            tc_fence_after();
            const uint64_t ka = operand(ring_k + st * G::kStage, TileGeo<D>::kGroup, 0);
            const uint32_t to = tmem + 128 * b + 32 * split.group(k);
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint64_t at = (uint64_t)(TileGeo<D>::step(x) >> 4);
                    mma_ss(to, ka + at, qb + at, is, x > 0);
                }
                tc_commit(smem_u32(&sh->rk.empty[st]));
                tc_commit(smem_u32(&sh->s_full[split.bar(k)][b]));
            }
            __syncwarp();
            if (++st == G::kKeys) st = 0, ++round;
        }
        if (elect_one()) qs.each([&](int x, uint32_t) { tc_commit(smem_u32(&sh->q_empty[x])); });
        __syncwarp();
        qs.done();
    }
}

template <int D>
__device__ void narrow_outputs(const AttnParams& p, const Ctl& ctl, NarrowShared<D>* sh, uint32_t sp, uint32_t ring_v, uint32_t tmem) {
    using G = NarrowGeo<D>;
    Weights weights;
    uint32_t st = 0, round = 0;
    int turn = 0;
    for (uint32_t i = 0;; ++i) {
        const int rows = sh->pieces.get(ctl, i);
        if (rows == 0) return;
        const PieceInfo& c = sh->pieces.at(i);
        const int n = uniform(c.n), first_tail = c.first_tail(7), keys = uniform(c.end - c.key0);
        const Split split(rows, n, turn);
        const uint32_t io = instruction(32 * split.used, 1, 1);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const int k = t & (split.tiles() - 1), r = t >> split.log_tiles, b = r & 1, g = split.group(k);
            wait(ctl, smem_u32(&sh->rv.full[st]), round & 1);
            if (t >= first_tail) {  // while the weights are worked out
                if (clean_values<D>(ring_v + st * G::kStage, max(c.ctx - c.key0 - t * kTile, 0), keys - t * kTile, threadIdx.x & 31, 32))
                    *reinterpret_cast<volatile uint32_t*>(&sh->poison[i % kPieces]) = i + 1;
                fence_async_smem();
                __syncwarp();
            }
            for (int x = 0; x < split.used; ++x) weights.wait_for(ctl, sh, 2 * (g + x) + b);
            tc_fence_after();
            // 64 columns of V have no second block: the upper half of the outputs repeats the lower one
            const uint64_t va = operand(ring_v + st * G::kStage, TileGeo<D>::kGroup, D == 128 ? 1024 : 0);
            const uint64_t pb = operand(sp + (g >> 1) * G::kBlock + (g & 1) * 64, 1024, G::kBlock);
            const uint32_t to = tmem + 256 + 32 * g, more = r > 0;
            const int steps = tile_steps(keys - t * kTile);
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < kTile / 16; ++x) {
                    if (x < steps)
                        mma_ss(to, va + (uint64_t)((x * 2 * TileGeo<D>::kGroup) >> 4), pb + (uint64_t)((x * 2048) >> 4), io, x > 0 ? 1u : more);
                }
                tc_commit(smem_u32(&sh->rv.empty[st]));
                tc_commit(smem_u32(&sh->o_full[split.bar(k)][b]));
                mbar_arrive(smem_u32(&sh->o_full[split.bar(k)][b]));  // orders the piece's poison before it
            }
            __syncwarp();
            if (++st == G::kValues) st = 0, ++round;
        }
        sh->pieces.done(i);
    }
}

// ---- softmax ----

// 32 lanes' sums of 32 columns: lane k gets column k's.
__device__ __forceinline__ float sum_columns(float* v, int lane) {
#pragma unroll
    for (int h = 16; h > 0; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float send = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, h);
        }
    }
    return v[0];
}

__device__ __forceinline__ void ld8(uint32_t addr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void st8(uint32_t addr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "r"(addr)
                 : "memory");
}

// Whether any thread of a group's four warps says yes.
__device__ __forceinline__ bool group_any(int g, bool yes) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)yes), "r"(2 + g)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int g) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(2 + g) : "memory");
}

// What the row's nodes with a NaN or infinity in column d of their values add to it.
__device__ __forceinline__ float poison_of(const AttnParams& p, const PieceInfo& c, int node, int d) {
    const int j0 = max(0, c.key0 - c.ctx), j1 = min(c.end, c.key0 + c.n * kTile) - c.ctx;
    float sum = 0.0f;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        if (!attn_sees(p, (long long)c.node0 + node, node, j)) continue;
        const int pos = c.ctx + j;
        const size_t page = attn_page(p, c.seq, pos >> p.page_shift);
        const uint32_t b = __ldg(static_cast<const uint16_t*>(p.v_cache) +
                                 ((page * p.Hkv + c.hkv) * p.page_size + (pos & (p.page_size - 1))) * p.D + d);
        if ((b & 0x7f80u) == 0x7f80u) sum += __uint_as_float(b << 16);
    }
    return sum;
}

template <int D, bool kPlanned>
__device__ void narrow_softmax(const AttnParams& p, const Ctl& ctl, NarrowShared<D>* sh, unsigned char* spw, uint32_t tmem) {
    using G = NarrowGeo<D>;
    const int tid = threadIdx.x, lane = tid & 31, g = tid >> 7, key = tid & 127, quad = (tid >> 5) & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const float scale = p.scale2 != 0.0f ? p.scale2 : 1e-30f;  // 0: equal weights, and what is not seen stays so
    float* my_m = &sh->m[32 * g];
    // A group's 32 columns of the weights: 64 bytes of each key's 128-byte line, swizzled. Sixteen places of the first
    // eight keys' also carry 4 x 32 floats (one of each warp and column) between products.
    auto place = [&](int group, int wq) {
        const int x = 8 * wq + (lane >> 2), k = x >> 2;
        return reinterpret_cast<float*>(spw + (group >> 1) * G::kBlock + k * 128 + ((((group & 1) * 4 + (x & 3)) ^ (k & 7)) << 4)) +
               (lane & 3);
    };
    Uses all_uses{};
    int pending = 0, turn = 0;
    for (uint32_t piece = 0;; ++piece) {
        const int rows = sh->pieces.get(ctl, piece);
        const PieceInfo& c = sh->pieces.at(piece);
        const int n = c.n;
        // All warps of a group take the piece or none, and all groups where it is theirs together: they meet at barriers below.
        // Every group leaves through the barrier of all.
        const bool stop = group_any(g, rows == 0);
        const Split split(rows, n, turn);
        if ((stop || !split.solo) && rows_any<kSoftThreads>(stop)) break;
        const Uses uses = all_uses;
        all_uses.add(n, split);
        if (!kPlanned && c.join > 0) {
            if (tid == 0) sh->pieces.pending[pending] = c;
            ++pending;
        }
        if (split.solo && g != split.first) {
            sh->pieces.done(piece);
            continue;
        }
        const int first_tail = c.first_tail(7);
        const int k = split.solo ? 0 : g >> split.log_chunks, chunk = split.solo ? 0 : g & (split.chunks() - 1), bar = split.bar(k);
        my_m[lane] = kNone;  // all four warps: each finds it there
        __syncwarp();
        float l[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) l[e] = 0.0f;
        // this lane's row of the group's chunk
        const int my_row = c.row0 + min(32 * chunk + lane, rows - 1), my_node = attn_node(p, my_row);
        const int rounds = chunk < split.used ? split.rounds(n, k) : 0;
#pragma unroll 1
        for (int i = 0; i < rounds; ++i) {
            const int tt = (i << split.log_tiles) + k, b = i & 1;
            const bool tail = tt >= first_tail;
            // the product that read the group's weights last
            auto weights_free = [&] {
                if (i > 0) wait(ctl, smem_u32(&sh->o_full[bar][b ^ 1]), uses.parity(bar, b ^ 1, (i - 1) / 2));
            };
            wait(ctl, smem_u32(&sh->s_full[bar][b]), uses.parity(bar, b, i / 2));
            tc_fence_after();
            uint32_t seen = 0xffffffffu;  // rows that see this thread's key
            if (tail) {
                const int ctx = c.ctx, keys = c.end, pos0 = c.key0 + tt * kTile, pos = pos0 + key;
                if (!p.mask) {
                    // a chain: node j is seen by the rows from j * gq on
                    seen = pos < ctx ? 0xffffffffu : (pos < keys ? ~low_bits((pos - ctx) * p.gq - c.row0 - 32 * chunk) : 0u);
                } else {
                    // lane e works out which of the warp's 32 keys row e sees; then every lane picks its key's bits
                    const uint32_t row_sees = seen32(p, p.mask + (long long)(c.node0 + my_node) * p.words, my_node, ctx, keys, pos0 + 32 * quad);
                    seen = 0;
#pragma unroll 8
                    for (int e = 0; e < 32; ++e) seen |= ((__shfl_sync(0xffffffffu, row_sees, e) >> lane) & 1u) << e;
                }
            }
            const uint32_t t_s = tmem + lanes + 128 * b + 32 * g;
            float z[32];  // scores, then arguments of the exponential
            bool move = i == 0;  // whether references have to move: always in the first tile
#pragma unroll 1
            for (bool moved = false;;) {
                if (move) {
                    // the columns' maxima: lane e has the warp's of column e, the four meet in the buffer that the
                    // weights are about to fill
                    float mine = kNegInf;
#pragma unroll 1
                    for (int e = 0; e < 32; e += 8) {
                        float v[8];
                        ld8(t_s + e, v);
                        tc_wait_ld();
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float r = (seen >> (e + x)) & 1u ? v[x] * scale : kNegInf;
                            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(r));
                            mine = lane == e + x ? r : mine;
                        }
                    }
                    weights_free();
                    *place(g, quad) = mine;
                    group_sync(g);
                    const float best = fmaxf(fmaxf(*place(g, 0), *place(g, 1)), fmaxf(*place(g, 2), *place(g, 3)));
                    const float old = my_m[lane];
                    const float to = best - old > 8.0f ? best : old;
                    const float fac = to == old ? 1.0f : ex2(old - to);
                    group_sync(g);    // old references and maxima have been read
                    my_m[lane] = to;  // all four warps: each finds it there from now on
                    __syncwarp();
                    if (i > 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) l[e] *= __shfl_sync(0xffffffffu, fac, e);
                        tc_fence_after();
#pragma unroll 1
                        for (int e = 0; e < 32; e += 8) {
                            float o[8];
                            ld8(tmem + lanes + 256 + 32 * g + e, o);
                            tc_wait_ld();
#pragma unroll
                            for (int x = 0; x < 8; ++x) o[x] *= __shfl_sync(0xffffffffu, fac, e + x);
                            st8(tmem + lanes + 256 + 32 * g + e, o);
                        }
                        tc_wait_st();
                    }
                    moved = true;
                }
                ld32(t_s, z);
                tc_wait_ld();
                float top = kNegInf;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(my_m + e);
                    z[e] = fmaf(z[e], scale, -m.x);
                    z[e + 1] = fmaf(z[e + 1], scale, -m.y);
                    z[e + 2] = fmaf(z[e + 2], scale, -m.z);
                    z[e + 3] = fmaf(z[e + 3], scale, -m.w);
                    if (tail) {
#pragma unroll
                        for (int x = e; x < e + 4; ++x) z[x] = (seen >> x) & 1u ? z[x] : kNegInf;
                    }
                    asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(z[e]), "f"(z[e + 1]));
                    asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(z[e + 2]), "f"(z[e + 3]));
                }
                if (moved) break;
                move = group_any(g, top > 8.0f);
                if (!move) break;
            }
            // this key's weights of 32 rows: four 16-byte places of its line
            weights_free();
            unsigned char* line = spw + (g >> 1) * G::kBlock + key * 128;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t pk[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float a = ex2(z[e + 2 * x]), d = ex2(z[e + 2 * x + 1]);
                    l[e + 2 * x] += a;
                    l[e + 2 * x + 1] += d;
                    pk[x] = pack_bf16(a, d);
                }
                *reinterpret_cast<uint4*>(line + ((((g & 1) * 4 + e / 8) ^ (key & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[g][b]));
        }
        // the group's last product; then the statistics meet where the weights were
        if (rounds > 0) {
            const int i = rounds - 1;
            wait(ctl, smem_u32(&sh->o_full[bar][i & 1]), uses.parity(bar, i & 1, i / 2));
        }
        *place(g, quad) = sum_columns(l, lane);
        __syncwarp();
        const bool poisoned = *reinterpret_cast<volatile uint32_t*>(&sh->poison[piece % kPieces]) == piece + 1;
        const bool poison = split.solo ? group_any(g, poisoned) : rows_any<kSoftThreads>(poisoned);
        tc_fence_after();
        if (chunk < split.used) {
            // the groups of a chunk join its rows, each a part of them: lane e has row e's factors
            float m = kNone, sum = 0.0f, f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (x < split.tiles()) m = fmaxf(m, sh->m[32 * (split.group(x) + chunk) + lane]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                f[x] = 0.0f;
                if (x >= split.tiles()) continue;
                const int from = split.group(x) + chunk;
                f[x] = ex2(sh->m[32 * from + lane] - m);
                sum = fmaf((*place(from, 0) + *place(from, 1)) + (*place(from, 2) + *place(from, 3)), f[x], sum);
            }
            if (c.whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int x = 0; x < 4; ++x) f[x] *= inv;
            }
            const int orow = (c.node0 + my_node) * p.Hq + c.hkv * p.gq + (my_row - my_node * p.gq);
            if (k == 0 && quad == 0 && 32 * chunk + lane < rows) {
                if (!c.whole)
                    c.ml[32 * chunk + lane] = make_float2(m, sum);
                else if (p.lse)
                    p.lse[orow] = attn_lse(m, sum);
            }
            const int part = 32 >> split.log_tiles, d = quad * 32 + lane, count = min(32, rows - 32 * chunk);
            if (quad * 32 < D) {  // otherwise repeated outputs
                // rows of the result, or of the slot
                const bool whole = c.whole;
                const int row_to = whole ? orow : 32 * chunk + lane, size = whole ? 2 : 4;
                char* base = (whole ? static_cast<char*>(p.out) : reinterpret_cast<char*>(c.o)) + d * size;
#pragma unroll 1
                for (int e = k * part; e < (k + 1) * part && e < count; e += 8) {
                    float v[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[y] = 0.0f;
#pragma unroll 1
                    for (int x = 0; x < split.tiles() && x < n; ++x) {
                        float o[8];
                        ld8(tmem + lanes + 256 + 32 * (split.group(x) + chunk) + e, o);
                        tc_wait_ld();
                        const float fx = x < 2 ? (x == 0 ? f[0] : f[1]) : (x == 2 ? f[2] : f[3]);
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[y] = fmaf(o[y], __shfl_sync(0xffffffffu, fx, e + y), v[y]);
                    }
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        char* to = base + (long long)__shfl_sync(0xffffffffu, row_to, e + y) * (D * size);
                        if (e + y >= count) continue;
                        if (whole)
                            *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(v[y]);
                        else
                            *reinterpret_cast<float*>(to) = v[y];
                    }
                }
                if (poison) {
#pragma unroll 1
                    for (int e = k * part; e < (k + 1) * part && e < count; ++e) {
                        const int row = c.row0 + 32 * chunk + e, node = attn_node(p, row);
                        const float v = poison_of(p, c, node, d);
                        if (v == 0.0f) continue;
                        const size_t to = (size_t)(c.node0 + node) * p.Hq + c.hkv * p.gq + (row - node * p.gq);
                        if (c.whole) {
                            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + to * D + d;
                            *o = __float2bfloat16_rn(__bfloat162float(*o) + v);
                        } else {
                            c.o[(size_t)(32 * chunk + e) * D + d] += v;
                        }
                    }
                }
            }
        }
        tc_fence_before();
        sh->pieces.done(piece);
        // everything has been read: the next piece may write over it
        if (split.solo)
            group_sync(g);
        else
            rows_sync<kSoftThreads>();
    }
    if (!kPlanned && pending > 0)  // behind the barrier of the loop's end
        attn_join_last<1, D, 1, 4>(p, sh->pieces.pending, pending, tid, kSoftThreads, sh->pieces.last, [] { rows_sync<kSoftThreads>(); });
}

template <int D, bool kPlanned>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_narrow_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using G = NarrowGeo<D>;
    extern __shared__ unsigned char dyn[];
    __shared__ NarrowShared<D> shared;
    NarrowShared<D>* sh = &shared;
    unsigned char* sq = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    unsigned char* spw = sq + G::kStage;
    const uint32_t ring_k = smem_u32(spw + G::kWeights), ring_v = ring_k + G::kKeys * G::kStage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh->rk.init(1);
        sh->rv.init(1);
        sh->pieces.init(19);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh->q_full[i]), 32);
            mbar_init(smem_u32(&sh->q_empty[i]), 1);
        }
        for (int i = 0; i < kPieces; ++i) sh->poison[i] = 0;
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_u32(&sh->s_full[i >> 1][i & 1]), 1);
            mbar_init(smem_u32(&sh->o_full[i >> 1][i & 1]), 2);
            mbar_init(smem_u32(&sh->p_full[i >> 1][i & 1]), 4);
        }
        sh->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 17) {
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
    // 640 threads start with 96 registers each; the softmax's sixteen warps go on with 104 and the other four with
    // 64 (4 x 104 + 64 = 5 x 96)
    if (warp < 16) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        narrow_softmax<D, kPlanned>(p, ctl, sh, spw, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 17)
            narrow_scores<D>(p, ctl, sh, smem_u32(sq), ring_k, tmem);
        else if (warp == 19)
            narrow_outputs<D>(p, ctl, sh, smem_u32(spw), ring_v, tmem);
        else
            narrow_fill<D, kPlanned>(p, warp == 16, warp == 16 ? &mk : &mv, ctl, sh, smem_u32(sq), warp == 16 ? ring_k : ring_v, lane);
    }
    tc_fence_before();
    __syncthreads();
    settle(ctl);
    if (warp == 17) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

template <int D>
static cudaError_t launch_narrow_t(const AttnParams& p, cudaStream_t st) {
    return launch_tc(p.planned ? attn_narrow_kernel<D, true> : attn_narrow_kernel<D, false>, kTcThreads, NarrowGeo<D>::kSmem, p, st);
}

cudaError_t launch_attn_narrow(const AttnParams& p, cudaStream_t st) {
    return p.D == 64 ? launch_narrow_t<64>(p, st) : launch_narrow_t<128>(p, st);
}

}  // namespace smcsd
