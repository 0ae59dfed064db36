// attn_plan.cuh -- how the work of tree_attention is cut up, shared by its kernels.
//
// Items. An item is a run of nodes (rows of q) that reads one run of keys of one page table row:
// for a group of N > 1 sequences whose tables start with the same pages, one item of all the group's
// nodes over those shared keys; and for every sequence one item of its own nodes over the keys that
// are left (all of them without sharing), the drafted nodes at the end among them. An item has
// Hkv x nrb units (a key/value head and a block of at most RB rows, a row being a node and one of the
// Hq/Hkv query heads that share the head), each of `tiles` tiles of keys.
//
// Cut. All tiles of all units stand in one line, each of them on as many places as its unit's rows make it cost, and before each
// unit's tiles as many empty places as beginning and ending a unit costs: W places (below 2^31). Block c of ncta has W / ncta
// of them, the first W % ncta blocks one more, and takes the tiles that begin there: shares of equal cost whatever the lengths
// and the rows are. Where a block would not get a tile's places, all tiles count one (AttnCost). Where a cut falls inside a unit, or a
// row has a shared and an own unit, the pieces leave (sum, max, weighted values) in a slot. Without groups only a block's first
// and last piece can be part of a unit: block c has slots 2 c (a unit that began before it) and 2 c + 1 (one that ends behind
// it). With groups a piece of unit u in block c has slot u + c (both rise along the line and one of them rises from piece to
// piece, so no two pieces share a slot). Without the planning kernel the last block to finish a unit's pieces joins them, in
// the order of the line; with it a kernel of its own joins a row's pieces. The kernels exist once for each of the
// two: what a call does not come to costs it all the same, since their code is longer than what an SM holds of it at a time.
//
// Who works the line out. Without groups and for up to 1024 sequences a warp of each block does, from the lengths
// alone (a few loads, all in flight together; a planning kernel before it and the loads of its results took 5 us of a
// call's 17). Otherwise the planning kernel writes the items down.
#pragma once

#include <cuda_bf16.h>

#include "smcsd_internal.cuh"

namespace smcsd {

struct __align__(16) AttnItem {
    int node0, nodes;   // rows of q
    int key0, tiles;    // first key, key tiles of each unit
    int nrb, per;       // row blocks, rows in each of them (the last one may be shorter)
    int seq, unit0;     // page table row; number of the first unit
    int cum;            // first place on the line
    int keys;           // keys that a group shares (key0 of its sequences)
    int pad[2];
};

struct AttnHead {  // written by the planning kernel
    int ncta, base, rest;  // W = ncta * base + rest
    int units_shared;      // units of shared items, which are the first ones
    int weighted;          // AttnCost
};

// Blocks on the line: one or two for each SM, of which the GPU has 152 and a kernel uses no more than kAttnMaxSm. The scratch is
// sized for them.
constexpr int kAttnMaxSm = 160, kAttnMaxCta = 2 * kAttnMaxSm;
static_assert(kAttnMaxCta <= kFrontArrivals, "a block's counter in the workspace's front");
constexpr int kAttnWarpPlan = 1024;  // sequences whose places on the line a warp works out
inline bool attn_planned(int S, int N) { return N > 1 || S > kAttnWarpPlan; }

struct AttnLayout {
    size_t head;     // AttnHead
    size_t item;     // AttnItem [G + S]
    size_t shared;   // int [G] keys shared by a group
    size_t slot_g;   // pieces of shared units: float [slots][rows_g][D], then float2 [slots][rows_g]
    size_t slot_s;   // pieces of own units
    size_t ml_g, ml_s;
    int rows_g, rows_s;
    size_t total;
};

inline int attn_blocks(long long rows, int rb) { return (int)((rows + rb - 1) / rb); }

inline AttnLayout attn_layout(int S, int N, int T, int gq, int Hkv, int D, int RB, int ncta) {
    AttnLayout L{};
    const size_t G = N > 1 ? (size_t)S / N : 0;
    size_t o = kFrontBytes;
    L.head = o;
    o = align256(o + sizeof(AttnHead));
    L.item = o;
    o = align256(o + sizeof(AttnItem) * (G + S));
    L.shared = o;
    o = align256(o + 4 * G);
    const long long rs = (long long)T * gq, rg = rs * N;
    L.rows_s = (int)(rs < RB ? rs : RB);
    L.rows_g = (int)(rg < RB ? rg : RB);
    const size_t us = G ? (size_t)S * Hkv * attn_blocks(rs, RB) + ncta : 2 * (size_t)ncta;
    const size_t ug = G ? G * Hkv * attn_blocks(rg, RB) + ncta : 0;
    L.slot_s = o;
    o = align256(o + us * L.rows_s * D * 4);
    L.ml_s = o;
    o = align256(o + us * L.rows_s * 8);
    L.slot_g = o;
    o = align256(o + ug * L.rows_g * D * 4);
    L.ml_g = o;
    o = align256(o + ug * L.rows_g * 8);
    L.total = o;
    return L;
}

struct AttnParams {
    const void* q;
    long long q_stride;
    const void* k_cache;
    const void* v_cache;
    int num_pages, page_size, page_shift;
    const int32_t* table;
    int pages_per_seq;
    const int32_t* ctx_len;
    const int32_t* node_offsets;
    int S, N, G, T, R;  // G: groups with sharing looked for (0 if N == 1)
    const uint32_t* mask;
    int words;
    int Hq, Hkv, gq, D;
    float scale2;  // scale * log2(e)
    void* out;
    float* lse;
    void* ws;
    AttnLayout L;
    int log_tile, log_rb;  // keys of a tile, rows of a block
    int heavy, w_light, w_heavy, empty;  // places of a tile of up to `heavy` rows, of more, before a unit's tiles
    int empty_one;                       // the last where a tile has one place
    int ncta_max;
    FastDiv div_gq, div_cta;
    bool planned;  // by the planning kernel
};

__device__ __forceinline__ AttnHead* attn_head(const AttnParams& p) { return ws_ptr<AttnHead>(p.ws, p.L.head); }

// First row and number of nodes of sequence s; none (and an error) if the offsets do not fit.
__device__ __forceinline__ int attn_nodes(const AttnParams& p, int s, int& node0) {
    if (!p.node_offsets) {
        node0 = s * p.T;
        return p.T;
    }
    const int a = __ldg(p.node_offsets + s), b = __ldg(p.node_offsets + s + 1);
    node0 = a;
    if (a < 0 || b < a || b > p.R || b - a > p.T) {
        raise_error(p.ws, kErrRange);
        return 0;
    }
    return b - a;
}
// Tokens in the cache of sequence s, or -1 (and an error) if they and n new ones do not fit its table.
__device__ __forceinline__ int attn_ctx(const AttnParams& p, int s, int n) {
    const int c = __ldg(p.ctx_len + s);
    if (c < 0 || (long long)c + n > ((long long)p.pages_per_seq << p.page_shift)) {
        raise_error(p.ws, kErrRange);
        return -1;
    }
    return c;
}

struct AttnCut {  // W = ncta * base + rest
    int base, rest, ncta;
    __device__ __forceinline__ AttnCut() {}
    __device__ __forceinline__ AttnCut(const AttnParams& p, int W) {
        ncta = min(p.ncta_max, W);
        base = W < p.ncta_max ? 1 : (int)fast_div((uint32_t)W, p.div_cta);
        rest = W - base * ncta;
    }
    __device__ __forceinline__ int of(int c) const { return base * c + min(c, rest); }  // first place of block c
    __device__ __forceinline__ int block(int x) const {                                 // of place x
        const int first = rest * (base + 1);  // places of the longer shares
        const bool longer = x < first;
        return (longer ? 0 : rest) + (int)((unsigned)(longer ? x : x - first) / (unsigned)(longer ? base + 1 : base));
    }
};

// What tiles and units cost in places. `weighted` only where every block has at least a tile's places, so that each of the
// blocks between a unit's first and last tile has a tile of it.
struct AttnCost {
    int heavy, light_tile, heavy_tile, empty;
    __device__ __forceinline__ AttnCost() {}
    __device__ __forceinline__ AttnCost(const AttnParams& p, bool weighted)
        : heavy(p.heavy), light_tile(weighted ? p.w_light : 1), heavy_tile(weighted ? p.w_heavy : 1), empty(weighted ? p.empty : p.empty_one) {}
    __device__ __forceinline__ static bool fits(const AttnParams& p, long long W) { return W >= (long long)p.w_heavy * p.ncta_max; }
    __device__ __forceinline__ int tile(int rows) const { return rows > heavy ? heavy_tile : light_tile; }
    __device__ __forceinline__ int unit(int rows, int tiles) const { return tile(rows) * tiles + empty; }
    // the row blocks of one head
    __device__ __forceinline__ int head(const AttnParams& p, const AttnItem& it) const {
        return (it.nrb - 1) * unit(it.per, it.tiles) + unit(it.nodes * p.gq - (it.nrb - 1) * it.per, it.tiles);
    }
    __device__ __forceinline__ int item(const AttnParams& p, const AttnItem& it) const { return it.tiles > 0 ? p.Hkv * head(p, it) : 0; }
};

// Row blocks of an item, and its units.
__device__ __forceinline__ int attn_units(const AttnParams& p, AttnItem& it) {
    const int rows = it.nodes * p.gq, rb = 1 << p.log_rb;
    it.nrb = max(1, (rows + rb - 1) >> p.log_rb);
    it.per = max(1, min(rows, rb));
    if (it.nodes == 0 || it.tiles < 0) it.tiles = 0;
    return it.tiles > 0 ? p.Hkv * it.nrb : 0;
}

// A warp's search: the item that place x of the line lies in, 32 at a time (the last one that begins at or before it: items
// without tiles come before the one that has them).
__device__ __forceinline__ int attn_search(const AttnItem* items, int first, int n, int x, int lane) {
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool below = lane * step < n && __ldcg(&items[first + lane * step].cum) <= x;
        const int k = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
        n = min(step, n - k * step);
        first += k * step;
    }
    return first;
}

// One piece of a unit, as a block comes to it on its share of the line and hands it round in shared memory.
struct PieceInfo {
    float* o;  // its slot
    float2* ml;
    int join, counter;       // pieces of the unit, joined by the last to arrive (0: none are); its first block, its counter
    int node0, seq, hkv;     // first row of the item, page table row, key/value head
    int row0, rows;          // rows of the item in this block of rows (none: there are no more pieces)
    int key0, n;             // first key, key tiles
    int ctx, end;            // tokens in the cache and behind them the nodes; for keys that a group shares both are their end
    bool whole;              // all that its rows have to see: the result is written directly
    // first tile with a node or the end inside it (n or more: none; rounded down, below zero where nodes are all there is)
    __device__ __forceinline__ int first_tail(int log_size) const { return (ctx - key0) >> log_size; }
};

// A warp's walk along its block's share, with the items of the planning kernel or from the lengths alone.
template <bool kPlanned>
struct Walker {
    AttnCut cut;
    AttnCost cost;
    int x, end, item_end;
    int units_shared, ii;  // ii: number of the present item
    AttnItem it;
    int unit, hkv, rb, at, ctx;  // next unit of it, its head and block of rows, first place of what is left; its tokens in the cache
    // where the warp works the line out itself: 32 sequences at a time, one a lane
    AttnItem mine;
    int first, mine_end;  // the 32's first sequence, line after this lane's item

    // this lane's item of the 32
    __device__ __forceinline__ void load(const AttnParams& p, int lane) {
        const int s = first + lane;
        mine.nodes = mine.tiles = mine.node0 = 0;
        if (s < p.S) {
            mine.nodes = attn_nodes(p, s, mine.node0);
            const int c = attn_ctx(p, s, mine.nodes);
            if (c < 0) mine.nodes = 0;
            mine.tiles = mine.nodes > 0 ? (c + mine.nodes + (1 << p.log_tile) - 1) >> p.log_tile : 0;
        }
        attn_units(p, mine);
    }
    __device__ __forceinline__ void place(int at, int size, int lane) {
        int in = size;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += t;
        }
        mine_end = at + in;
        mine.cum = mine_end - size;
    }

    __device__ __forceinline__ void begin(const AttnParams& p, int lane) {
        const int cta = blockIdx.x;
        x = end = item_end = 0;
        units_shared = 0;
        if (kPlanned) {
            const AttnHead* h = attn_head(p);
            cut.base = h->base;
            cut.rest = h->rest;
            units_shared = h->units_shared;
            cost = AttnCost(p, h->weighted);
            if (cta >= h->ncta) return;
            x = item_end = cut.of(cta);
            end = cut.of(cta + 1);
            ii = attn_search(ws_ptr<AttnItem>(p.ws, p.L.item), 0, p.G + p.S, x, lane) - 1;
            return;
        }
        int W = 0, one = 0;
#pragma unroll 1
        for (first = 0; first < p.S; first += 32) {
            load(p, lane);
            W += __reduce_add_sync(0xffffffffu, AttnCost(p, true).item(p, mine));
            one += __reduce_add_sync(0xffffffffu, AttnCost(p, false).item(p, mine));
        }
        const bool weighted = AttnCost::fits(p, W);
        cost = AttnCost(p, weighted);
        W = weighted ? W : one;
        first -= 32;
        if (first == 0) {
            place(0, cost.item(p, mine), lane);
        } else {
            first = -32;  // next_item begins with the first 32
            mine_end = 0;
        }
        cut = AttnCut(p, W);
        if (cta >= cut.ncta) return;
        x = item_end = cut.of(cta);
        end = cut.of(cta + 1);
    }
    __device__ __forceinline__ void next_item(const AttnParams& p, int lane) {
        if (kPlanned) {
            it = ws_ptr<AttnItem>(p.ws, p.L.item)[++ii];
        } else {
            unsigned after;  // lanes whose items end behind x
            while ((after = __ballot_sync(0xffffffffu, mine_end > x)) == 0) {
                const int at = __shfl_sync(0xffffffffu, mine_end, 31);
                first += 32;
                load(p, lane);
                place(at, cost.item(p, mine), lane);
            }
            const int l = __ffs(after) - 1;
            it.node0 = __shfl_sync(0xffffffffu, mine.node0, l);
            it.nodes = __shfl_sync(0xffffffffu, mine.nodes, l);
            it.tiles = __shfl_sync(0xffffffffu, mine.tiles, l);
            it.cum = __shfl_sync(0xffffffffu, mine.cum, l);
            attn_units(p, it);
            it.unit0 = 0;
            it.key0 = 0;
            it.seq = ii = first + l;
        }
        item_end = it.cum + cost.item(p, it);
        ctx = ii >= p.G ? __ldg(p.ctx_len + it.seq) : 0;
    }
    // To the end, or the next unit.
    __device__ __forceinline__ void go_on(int to) {
        x = to;
        at = 0;
        ++unit;
        if (++rb == it.nrb) rb = 0, ++hkv;
    }
    // The next piece; false (and no rows) after the last one.
    __device__ __forceinline__ bool next(const AttnParams& p, PieceInfo& c, int lane) {
        c.rows = 0;
        int first, w, a, b, to;  // the unit's first tile's place, places of a tile, tiles from a to b, place behind them
#pragma unroll 1
        for (;; go_on(to)) {
            if (x >= end) return false;
            if (x >= item_end) {
                while (x >= item_end) next_item(p, lane);  // x is below W, so an item that holds it follows
                const int per_head = cost.head(p, it), per_unit = cost.unit(it.per, it.tiles);
                hkv = (int)((unsigned)(x - it.cum) / (unsigned)per_head);
                at = x - it.cum - hkv * per_head;
                rb = it.nrb == 1 ? 0 : min((int)((unsigned)at / (unsigned)per_unit), it.nrb - 1);
                at -= rb * per_unit;
                unit = hkv * it.nrb + rb;
            }
            c.row0 = rb * it.per;
            c.rows = min(it.nodes * p.gq - c.row0, it.per);
            w = cost.tile(c.rows);
            first = x - at + cost.empty;
            to = min(first + w * it.tiles, end);
            a = (int)((unsigned)(max(x - first, 0) + w - 1) / (unsigned)w);
            b = (int)((unsigned)(max(to - first, 0) + w - 1) / (unsigned)w);
            if (b > a) break;
            c.rows = 0;  // no tile of the unit begins on this share
        }
        const bool own = ii >= p.G;
        const int cta = blockIdx.x;
        c.node0 = it.node0;
        c.seq = it.seq;
        c.hkv = hkv;
        c.key0 = it.key0 + (a << p.log_tile);
        c.n = b - a;
        c.whole = own && it.key0 == 0 && c.n == it.tiles;
        c.ctx = own ? ctx : it.keys;
        c.end = own ? ctx + it.nodes : it.keys;
        c.join = 0;
        const int rows = own ? p.L.rows_s : p.L.rows_g;
        float* o = ws_ptr<float>(p.ws, own ? p.L.slot_s : p.L.slot_g);
        float2* ml = ws_ptr<float2>(p.ws, own ? p.L.ml_s : p.L.ml_g);
        size_t slot = (size_t)(it.unit0 + unit - (own ? units_shared : 0)) + cta;
        if (!kPlanned || p.G == 0) slot = 2 * cta + (a == 0);
        if (!kPlanned && !c.whole) {
            c.counter = cut.block(first);
            c.join = cut.block(first + (it.tiles - 1) * w) - c.counter + 1;
        }
        c.o = o + slot * rows * p.D;
        c.ml = ml + slot * rows;
        go_on(to);
        return true;
    }
};

// Both are off by at most 2^-22 (of the result; of lg2 between 1/2 and 2 absolutely), as much as exp2f is. Weights below 2^-126
// become zero.
__device__ __forceinline__ float attn_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float attn_lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Node and query head of row `row` of an item whose rows are those of key/value head hkv.
__device__ __forceinline__ int attn_node(const AttnParams& p, int row) { return (int)fast_div((uint32_t)row, p.div_gq); }
// log of a sum l of exp2(z - m)
__device__ __forceinline__ float attn_lse(float m, float l) { return l == 0.0f ? kNegInf : (m + attn_lg2(l)) * 0.69314718056f; }
template <int DT>
__device__ __forceinline__ void attn_store4(void* base, size_t i, float4 v) {
    if (DT == 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = v;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

// Pieces of one row, joined one after the other.
struct AttnJoin {
    float m = kNegInf, l = 0.0f;
    float4 acc = make_float4(0, 0, 0, 0);
    __device__ __forceinline__ void add(float2 ml, float4 v) {
        if (ml.y == 0.0f) return;  // saw nothing
        const float mx = fmaxf(m, ml.x);
        const float base = mx == kNegInf ? 0.0f : mx;
        const float fa = l == 0.0f ? 0.0f : attn_ex2(m - base), fb = attn_ex2(ml.x - base);
        l = l * fa + ml.y * fb;
        acc.x = fmaf(acc.x, fa, v.x * fb);
        acc.y = fmaf(acc.y, fa, v.y * fb);
        acc.z = fmaf(acc.z, fa, v.z * fb);
        acc.w = fmaf(acc.w, fa, v.w * fb);
        m = mx;
    }
    template <int DT, int D>
    __device__ __forceinline__ void store(const AttnParams& p, size_t orow, int col) const {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        attn_store4<DT>(p.out, orow * D + col, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (col == 0 && p.lse) p.lse[orow] = attn_lse(m, l);
    }
};

// The counter of a unit is that of the block in which it is cut first (kFrontArrive).
// The block's threads, all of whose stores to the pieces' slots lie before a barrier: reports up to two pieces (a block's
// first and last) and joins the units that they complete. `s_last` is shared; sync() a barrier of these threads.
template <int DT, int D, int kRows, int kPieces, typename Sync>
__device__ __forceinline__ void attn_join_last(const AttnParams& p, const PieceInfo* piece, int count, int tid, int threads,
                                               volatile int* s_last, Sync sync) {
    if (tid < count) {
        unsigned* counter = ws_ptr<unsigned>(p.ws, kFrontArrive) + piece[tid].counter;
        const bool last = atom_add_release(counter, 1u) == (unsigned)piece[tid].join - 1;
        if (last) {
            fence_acquire();
            atomicExch(counter, 0u);
        }
        s_last[tid] = last;
    }
    sync();
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
        if (!s_last[k]) continue;
        const PieceInfo c = piece[k];
        const float* o = ws_ptr<float>(p.ws, p.L.slot_s);
        const float2* ml = ws_ptr<float2>(p.ws, p.L.ml_s);
        // kRows rows and kPieces pieces a thread at a time, to have enough loads in flight
        const int step = threads / (D / 4), col = (tid % (D / 4)) * 4;
#pragma unroll 1
        for (int r0 = tid / (D / 4); r0 < c.rows; r0 += kRows * step) {
            AttnJoin j[kRows];
#pragma unroll 1
            for (int x0 = 0; x0 < c.join; x0 += kPieces) {
                float2 s[kPieces][kRows];
                float4 v[kPieces][kRows];
#pragma unroll
                for (int x = 0; x < kPieces; ++x) {
                    const int k = min(x0 + x, c.join - 1);
                    const size_t slot = 2 * (size_t)(c.counter + k) + (k == 0);
#pragma unroll
                    for (int y = 0; y < kRows; ++y) {
                        const size_t at = slot * p.L.rows_s + min(r0 + y * step, c.rows - 1);
                        s[x][y] = __ldcg(ml + at);
                        v[x][y] = __ldcg(reinterpret_cast<const float4*>(o + at * D + col));
                        if (x0 + x >= c.join) s[x][y].y = 0.0f;
                    }
                }
#pragma unroll
                for (int x = 0; x < kPieces; ++x)
#pragma unroll
                    for (int y = 0; y < kRows; ++y) j[y].add(s[x][y], v[x][y]);
            }
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
                const int r = r0 + y * step, row = c.row0 + r, node = attn_node(p, row);
                if (r < c.rows) j[y].store<DT, D>(p, (size_t)(c.node0 + node) * p.Hq + c.hkv * p.gq + (row - node * p.gq), col);
            }
        }
    }
}

// Whether node t (of the sequence whose first row is row0) sees node j.
__device__ __forceinline__ bool attn_sees(const AttnParams& p, long long row, int t, int j) {
    if (!p.mask) return j <= t;
    return (__ldg(p.mask + row * p.words + (j >> 5)) >> (j & 31)) & 1u;
}

__device__ __forceinline__ int attn_page(const AttnParams& p, int seq, int j) {
    int id = __ldg(p.table + (long long)seq * p.pages_per_seq + j);
    if (id < 0 || id >= p.num_pages) {
        raise_error(p.ws, kErrRange);
        id = 0;
    }
    return id;
}

cudaError_t launch_attn_plan(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_simt(const AttnParams& p, cudaStream_t st);  // float32
cudaError_t launch_attn_wide(const AttnParams& p, cudaStream_t st);    // bf16, row blocks of 256
cudaError_t launch_attn_narrow(const AttnParams& p, cudaStream_t st);  // bf16, row blocks of 128
cudaError_t launch_attn_combine(const AttnParams& p, int dtype, cudaStream_t st);

}  // namespace smcsd
