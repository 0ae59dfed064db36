// attn_plan.cuh -- how the work of tree_attention is cut up, shared by its kernels.
//
// Items. An item is a run of nodes (rows of q) that reads one run of keys of one page table row:
// for a group of N > 1 sequences whose tables start with the same pages, one item of all the group's
// nodes over those shared keys; and for every sequence one item of its own nodes over the keys that
// are left (all of them without sharing), the drafted nodes at the end among them. An item has
// Hkv x nrb units (a key/value head and a block of at most RB rows, a row being a node and one of the
// Hq/Hkv query heads that share the head), each of `tiles` tiles of keys.
//
// Cut. All tiles of all units stand in one line, W of them (below 2^31). Block c of ncta takes W / ncta of them,
// the first W % ncta blocks one more: equal shares whatever the lengths are. Where a cut falls inside a unit, or a
// row has a shared and an own unit, the pieces leave (sum, max, weighted values) in a slot and the
// combining kernel joins them in a fixed order. A piece of unit u in block c has the number u + c:
// both rise along the line and one of them rises from piece to piece, so no two pieces share a number.
#pragma once

#include "smcsd_internal.cuh"

namespace smcsd {

struct __align__(16) AttnItem {
    int node0, nodes;   // rows of q
    int tile0, tiles;   // key tiles of each unit
    int nrb, per;       // row blocks, rows in each of them (the last one may be shorter)
    int seq, unit0;     // page table row; number of the first unit
    int cum;            // first tile on the line
    int pad[3];
};

struct AttnHead {  // written by the planning kernel
    int flag;      // error flag (first word of every workspace)
    unsigned done; // blocks of the planning kernel that have finished
    int ncta, base, rest;  // W = ncta * base + rest
    int units, units_shared;  // units, those of shared items among them (the first ones)
};

struct AttnLayout {
    size_t item;     // AttnItem [G + S]
    size_t shared;   // int [G] tiles shared by a group
    size_t slot_g;   // pieces of shared units: float [slots][rows_g][D], then float2 [slots][rows_g]
    size_t slot_s;   // pieces of own units
    size_t ml_g, ml_s;
    int rows_g, rows_s;
    size_t total;
};

// Every kernel that takes part has at most kAttnMaxCta blocks on the line.
constexpr int kAttnMaxCta = 1024;

__host__ __device__ inline int attn_blocks(long long rows, int rb) { return (int)((rows + rb - 1) / rb); }

inline AttnLayout attn_layout(int S, int N, int T, int gq, int Hkv, int D, int RB, int ncta) {
    AttnLayout L{};
    const size_t G = N > 1 ? (size_t)S / N : 0;
    size_t o = 256;
    L.item = o;
    o = align256(o + sizeof(AttnItem) * (G + S));
    L.shared = o;
    o = align256(o + 4 * G);
    const long long rs = (long long)T * gq, rg = rs * N;
    L.rows_s = (int)(rs < RB ? rs : RB);
    L.rows_g = (int)(rg < RB ? rg : RB);
    const size_t us = (size_t)S * Hkv * attn_blocks(rs, RB) + ncta;
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
    int tile, rb, ncta_max, min_tiles;
};

__device__ __forceinline__ AttnHead* attn_head(const AttnParams& p) { return static_cast<AttnHead*>(p.ws); }

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

__device__ __forceinline__ int attn_cut(const AttnHead* h, int c) { return h->base * c + min(c, h->rest); }
__device__ __forceinline__ int attn_cta_of(const AttnHead* h, int x) {
    const int first = h->rest * (h->base + 1);  // tiles of the longer shares
    return x < first ? x / (h->base + 1) : h->rest + (x - first) / h->base;
}

// A warp's search: the last of items [first, first + n) whose key is at most x (the first one's is), 32 at a time. With
// keys that rise along the line it is the one that x lies in, as items without tiles come before it.
template <typename Key>
__device__ __forceinline__ int attn_search(const AttnItem* items, int first, int n, int x, int lane, Key key) {
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool below = lane * step < n && key(items[first + lane * step]) <= x;
        const int k = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
        n = min(step, n - k * step);
        first += k * step;
    }
    return first;
}

// One piece of a unit, as a block walks along its share of the line.
struct AttnPiece {
    int node0, seq;        // first row of the item, page table row
    int hkv, row0, rows;   // key/value head; rows of the item in this block of rows
    int t0, t1;            // key tiles
    bool own;              // holds the sequence's own keys (and nodes), not a group's shared ones
    bool whole;            // all that its rows have to see: the result is written directly
    float* o;              // its slot otherwise
    float2* ml;
};

__device__ __forceinline__ AttnPiece attn_piece(const AttnParams& p, const AttnItem& it, bool own, int x, int end, int cta,
                                                int units_shared, int& next) {
    AttnPiece c;
    const int in = x - it.cum, u = in / it.tiles, t = in - u * it.tiles;
    c.node0 = it.node0;
    c.seq = it.seq;
    c.hkv = u / it.nrb;
    const int rb = u - c.hkv * it.nrb;
    c.row0 = rb * it.per;
    const int left = it.nodes * p.gq - c.row0;
    c.rows = left < it.per ? left : it.per;
    const int unit_end = x - t + it.tiles;
    next = unit_end < end ? unit_end : end;
    c.t0 = it.tile0 + t;
    c.t1 = c.t0 + (next - x);
    c.own = own;
    c.whole = own && it.tile0 == 0 && t == 0 && next == unit_end;
    const int unit = it.unit0 + u;
    if (own) {
        const size_t slot = (size_t)(unit - units_shared + cta);
        c.o = ws_ptr<float>(p.ws, p.L.slot_s) + slot * p.L.rows_s * p.D;
        c.ml = ws_ptr<float2>(p.ws, p.L.ml_s) + slot * p.L.rows_s;
    } else {
        const size_t slot = (size_t)(unit + cta);
        c.o = ws_ptr<float>(p.ws, p.L.slot_g) + slot * p.L.rows_g * p.D;
        c.ml = ws_ptr<float2>(p.ws, p.L.ml_g) + slot * p.L.rows_g;
    }
    return c;
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
