// serve_api.cu -- C ABI of the step around the verify (page tables and slots, cache writes, node
// masks, attention over the cache, logits): host-side argument checks and launches.
#include <math.h>

#include "attn_plan.cuh"
#include "serve_launch.cuh"
#include "smcsd.h"
#include "smcsd_launch.cuh"

using namespace smcsd;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? SMCSD_OK : SMCSD_ERR_CUDA; }
size_t elem_bytes(int dtype) { return dtype == SMCSD_F32 ? 4 : 2; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) return SMCSD_ERR_INVALID_ARG;
    if (((uintptr_t)ws & 255u) != 0 || ws_bytes < need) return SMCSD_ERR_WORKSPACE;
    return SMCSD_OK;
}

// log2 of a page size of 8 .. 256, or -1
int page_shift(int page_size) {
    for (int b = 3; b <= 8; ++b)
        if (page_size == 1 << b) return b;
    return -1;
}

// words of a row of n bits, and blocks of n tokens, are counted in 32 bits with their last one filled up
constexpr int kMostBits = 0x7fffffff - 4095;

bool nodes_ok(const int32_t* offsets, int S, int T, int R) {
    if (S <= 0 || T <= 0 || T > kMostBits || R <= 0) return false;
    return offsets || (long long)S * T == R;
}

// Sizes that tree_attention takes.
bool attn_sizes_ok(int S, int N, int T, int Hq, int Hkv, int D) {
    if (S <= 0 || N <= 0 || S % N || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return false;
    if (D != 64 && D != 128) return false;
    // rows of a group, and units, are counted in 32 bits
    const long long rows = (long long)T * (Hq / Hkv);
    return rows * N < (1ll << 30) && (long long)S * Hkv * (rows / 16 + 1) < (1ll << 30);
}

// float32: the FP32 pipes, 64 keys x 16 rows at a time. bf16: the tensor cores, 128 keys x up to 128 rows (narrow) or 256 (wide)
// at a time. The narrow kernel's time grows with a sequence's rows, the wide one's hardly does. With groups the shared units
// have N times the rows; how much is shared is not known here, and from D / 4 rows on the wide kernel gains more where much is
// than it loses where nothing is. Measured in us, narrow / wide:
//   64 sequences over 4096 tokens, D = 128: 32 rows 140 / 152, 64 rows 151 / 159, 96 rows 166 / 171, 112 rows 194 / 176, 128 rows 198 / 178
//   16 over 4096, D = 64: 64 rows 66.5 / 67.8, 100 rows 104 / 73
//   8 groups of 16 over 2048, D = 128, a share of 0, 0.5 and 0.9 of the context alike:
//     20 rows 141 / 154, 138 / 140, 96 / 100; 36 rows 156 / 163, 159 / 164, 154 / 127; 64 rows 168 / 173, 198 / 203, 223 / 165
//   16 groups of 4 over 4096, D = 128: 20 rows 145 / 150, 108 / 114, 86 / 82; 36 rows 154 / 155, 138 / 137, 159 / 108
//   8 groups of 16 over 2048, D = 64: 8 rows 185 / 201, 182 / 157, 109 / 113; 17 rows 199 / 211, 206 / 199, 148 / 138;
//     32 rows 206 / 214, 239 / 229, 182 / 166
enum AttnKind { kSimt, kNarrow, kWide };
constexpr int kSimtBlocksPerSm = 2;
// Places on the line (attn_plan.cuh): {rows from which a tile is heavy, of a light tile, of a heavy one, before a unit's tiles}.
// A narrow tile takes 142 us' worth with 32 rows, 158 with 64, 183 with 96, 224 with 128 (64 sequences over 4096 tokens); a wide one of one
// block of rows is shared out between the two streams. Measured: 64 chains of up to 21 nodes 165 us with equal tiles, 161 so, 177
// with 2 : 4; 8 groups of 16 particles, whose own units are short and run four at a time, 118 / 110 / 99.5 / 102 us with 1 / 2 / 3 / 4
// before a unit; 8 trees of up to 64 nodes 349 us with 1 : 2, 329 with 2 : 3, 341 with 3 : 4.
struct LineCost { int heavy, light_tile, heavy_tile, empty; };
constexpr LineCost kNarrowGroups{64, 2, 3, 3}, kNarrowCost{64, 2, 3, 6}, kWideCost{128, 2, 3, 6};

AttnKind kind_of(int dtype, int N, int T, int Hq, int Hkv, int D) {
    if (dtype == SMCSD_F32) return kSimt;
    const int most = N > 1 ? D / 4 : D == 128 ? 96 : 64;
    return (long long)T * (Hq / Hkv) <= most ? kNarrow : kWide;
}

int rows_of(AttnKind k) { return k == kSimt ? 16 : k == kNarrow ? 128 : 256; }
int blocks_of(AttnKind k, int sms) { return (sms < kAttnMaxSm ? sms : kAttnMaxSm) * (k == kSimt ? kSimtBlocksPerSm : 1); }

AttnLayout layout_of(AttnKind k, int S, int N, int T, int Hq, int Hkv, int D) {
    return attn_layout(S, N, T, Hq / Hkv, Hkv, D, rows_of(k), blocks_of(k, kAttnMaxSm));
}

}  // namespace

extern "C" int kv_slot_map(const int32_t* ctx_len, const int32_t* node_offsets, int S, int T, int R,
                           const int32_t* table_in, int32_t* table_out, int pages_per_seq,
                           int page_size, const int32_t* refcount_in, int32_t* refcount_out,
                           int num_pages, int64_t* slots, int32_t* copy_src, int32_t* copy_dst,
                           void* ws, size_t ws_bytes, void* stream) {
    if (!ctx_len || !table_in || !table_out || !refcount_in || !refcount_out || !slots || !copy_src || !copy_dst)
        return SMCSD_ERR_INVALID_ARG;
    if (table_in == table_out || refcount_in == refcount_out) return SMCSD_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (!nodes_ok(node_offsets, S, T, R) || pages_per_seq <= 0 || shift < 0 || num_pages <= 0)
        return SMCSD_ERR_INVALID_ARG;
    if ((long long)pages_per_seq * page_size > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, slot_map_bytes(S, num_pages));
    if (rc) return rc;
    SlotParams p{};
    p.ctx_len = ctx_len;
    p.n = Nodes{node_offsets, S, T, R};
    p.table_in = table_in;
    p.table_out = table_out;
    p.pages_per_seq = pages_per_seq;
    p.page_size = page_size;
    p.page_shift = shift;
    p.ref_in = refcount_in;
    p.ref_out = refcount_out;
    p.num_pages = num_pages;
    p.slots = slots;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.ws = ws;
    p.free_list = slot_map_free_list();
    p.demand = slot_map_demand(num_pages);
    return from_cuda(launch_slot_map(p, (cudaStream_t)stream));
}

extern "C" int kv_append(const void* k_new, const void* v_new, int dtype, int R, int Hkv, int D,
                         long long token_stride, const int64_t* slots, const int32_t* copy_src,
                         const int32_t* copy_dst, const int32_t* ctx_len, int S, void* k_cache,
                         void* v_cache, int page_size, int num_pages, void* ws, size_t ws_bytes,
                         void* stream) {
    if (dtype != SMCSD_F32 && dtype != SMCSD_BF16) return SMCSD_ERR_DTYPE;
    if (!k_new || !v_new || !slots || !k_cache || !v_cache) return SMCSD_ERR_INVALID_ARG;
    if ((copy_src == nullptr) != (copy_dst == nullptr) || (copy_src && (!ctx_len || S <= 0)))
        return SMCSD_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (R <= 0 || Hkv <= 0 || D <= 0 || shift < 0 || num_pages <= 0) return SMCSD_ERR_INVALID_ARG;
    const size_t b = elem_bytes(dtype);
    if ((D * b) % 16 || token_stride < (long long)Hkv * D || (token_stride * b) % 16) return SMCSD_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache))
        return SMCSD_ERR_INVALID_ARG;
    if ((long long)Hkv * D > (1 << 24)) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    AppendParams p{};
    p.k_new = k_new;
    p.v_new = v_new;
    p.token_vecs = (long long)(token_stride * b / 16);
    p.R = R;
    p.Hkv = Hkv;
    p.row_vecs = (int)(D * b / 16);
    p.slots = slots;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.ctx_len = ctx_len;
    p.S = S;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.page_size = page_size;
    p.page_shift = shift;
    p.num_pages = num_pages;
    p.ws = ws;
    return from_cuda(launch_append(p, (cudaStream_t)stream));
}

extern "C" int tree_mask(const int32_t* parents, const int32_t* node_offsets, int S, int T, int R,
                         uint32_t* mask, void* ws, size_t ws_bytes, void* stream) {
    if (!parents || !mask || !nodes_ok(node_offsets, S, T, R)) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    MaskParams p{parents, Nodes{node_offsets, S, T, R}, mask, (T + 31) / 32, ws};
    return from_cuda(launch_tree_mask(p, (cudaStream_t)stream));
}

extern "C" size_t tree_attention_workspace_size(int S, int N, int T, int Hq, int Hkv, int D) {
    if (!attn_sizes_ok(S, N, T, Hq, Hkv, D)) return 0;
    const size_t a = layout_of(kSimt, S, N, T, Hq, Hkv, D).total,
                 b = layout_of(kind_of(SMCSD_BF16, N, T, Hq, Hkv, D), S, N, T, Hq, Hkv, D).total;
    return a > b ? a : b;
}

extern "C" int tree_attention(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                              int dtype, int num_pages, int page_size, const int32_t* table,
                              int pages_per_seq, const int32_t* ctx_len, const int32_t* node_offsets,
                              int S, int N, int T, int R, const uint32_t* mask, int Hq, int Hkv, int D,
                              float scale, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (dtype != SMCSD_F32 && dtype != SMCSD_BF16) return SMCSD_ERR_DTYPE;
    if (!q || !k_cache || !v_cache || !table || !ctx_len || !out) return SMCSD_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (!nodes_ok(node_offsets, S, T, R) || !attn_sizes_ok(S, N, T, Hq, Hkv, D)) return SMCSD_ERR_INVALID_ARG;
    if (num_pages <= 0 || shift < 0 || pages_per_seq <= 0 || !isfinite(scale)) return SMCSD_ERR_INVALID_ARG;
    if ((long long)pages_per_seq * page_size > 0x3fffffffLL || (long long)R * Hq > 0x7fffffffLL)
        return SMCSD_ERR_INVALID_ARG;
    const size_t b = elem_bytes(dtype);
    if (q_stride < (long long)Hq * D || (q_stride * b) % 16) return SMCSD_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, tree_attention_workspace_size(S, N, T, Hq, Hkv, D));
    if (rc) return rc;
    AttnParams p{};
    p.q = q;
    p.q_stride = q_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.page_shift = shift;
    p.table = table;
    p.pages_per_seq = pages_per_seq;
    p.ctx_len = ctx_len;
    p.node_offsets = node_offsets;
    p.S = S;
    p.N = N;
    p.G = N > 1 ? S / N : 0;
    p.T = T;
    p.R = R;
    p.mask = mask;
    p.words = (T + 31) / 32;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.gq = Hq / Hkv;
    p.D = D;
    p.scale2 = (float)((double)scale * 1.4426950408889634074);
    p.out = out;
    p.lse = lse;
    p.ws = ws;
    cudaStream_t st = (cudaStream_t)stream;
    const AttnKind kind = kind_of(dtype, N, T, Hq, Hkv, D);
    // all places of all units are numbered in 32 bits
    const long long units = (long long)S * Hkv * attn_blocks((long long)T * p.gq, rows_of(kind)) +
                            (long long)p.G * Hkv * attn_blocks((long long)N * T * p.gq, rows_of(kind));
    const long long keys = (long long)pages_per_seq * page_size, places = kind == kSimt ? (keys + 63) / 64 : 3 * ((keys + 127) / 128) + 6;
    if (units * places > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;
    p.L = layout_of(kind, S, N, T, Hq, Hkv, D);
    p.log_tile = kind == kSimt ? 6 : 7;
    p.log_rb = kind == kSimt ? 4 : kind == kNarrow ? 7 : 8;
    const LineCost cost = kind == kSimt ? LineCost{0, 1, 1, 0} : kind == kWide ? kWideCost : p.G > 0 ? kNarrowGroups : kNarrowCost;
    p.heavy = cost.heavy;
    p.w_light = cost.light_tile;
    p.w_heavy = cost.heavy_tile;
    p.empty = cost.empty;
    p.empty_one = kind == kSimt ? 0 : 1;
    p.div_gq = make_fastdiv((uint32_t)p.gq);
    p.ncta_max = blocks_of(kind, device_sm_count());
    p.div_cta = make_fastdiv((uint32_t)p.ncta_max);
    p.planned = attn_planned(S, N);
    cudaError_t e = p.planned ? launch_attn_plan(p, st) : cudaSuccess;
    if (e == cudaSuccess)
        e = kind == kSimt ? launch_attn_simt(p, st) : kind == kNarrow ? launch_attn_narrow(p, st) : launch_attn_wide(p, st);
    if (e == cudaSuccess && p.planned) e = launch_attn_combine(p, dtype, st);
    return from_cuda(e);
}

extern "C" int logits_process(const void* logits, void* out, int dtype, int R, int V, int S, int T,
                              const int32_t* node_offsets, const int32_t* node_tokens,
                              const uint32_t* mask, const int32_t* hist_tokens,
                              const int32_t* hist_offsets, int n_hist, const float* repetition,
                              const float* presence, const float* frequency,
                              const int32_t* bias_tokens, const float* bias_values,
                              const int32_t* bias_offsets, int n_bias, const uint32_t* allowed,
                              void* ws, size_t ws_bytes, void* stream) {
    if (dtype != SMCSD_F32 && dtype != SMCSD_BF16) return SMCSD_ERR_DTYPE;
    if (!logits || !out || V <= 0 || V > kMostBits || !nodes_ok(node_offsets, S, T, R)) return SMCSD_ERR_INVALID_ARG;
    if (S > 65535) return SMCSD_ERR_INVALID_ARG;
    if ((hist_tokens == nullptr) != (hist_offsets == nullptr)) return SMCSD_ERR_INVALID_ARG;
    if ((bias_tokens == nullptr) != (bias_values == nullptr) || (bias_tokens == nullptr) != (bias_offsets == nullptr))
        return SMCSD_ERR_INVALID_ARG;
    if (n_hist < 0 || n_bias < 0) return SMCSD_ERR_INVALID_ARG;
    if (mask && !node_tokens) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    LogitsParams p{};
    p.logits = logits;
    p.out = out;
    p.n = Nodes{node_offsets, S, T, R};
    p.V = V;
    p.vec = aligned16(logits) && aligned16(out) && ((size_t)V * elem_bytes(dtype)) % 16 == 0;
    p.node_tokens = node_tokens;
    p.mask = mask;
    p.words = (T + 31) / 32;
    p.hist_tokens = hist_tokens;
    p.hist_offsets = hist_offsets;
    p.n_hist = n_hist;
    p.n_bias = n_bias;
    p.repetition = repetition;
    p.presence = presence;
    p.frequency = frequency;
    p.bias_tokens = bias_tokens;
    p.bias_values = bias_values;
    p.bias_offsets = bias_offsets;
    p.allowed = allowed;
    p.allowed_words = (V + 31) / 32;
    p.ws = ws;
    return from_cuda(launch_logits(p, dtype, (cudaStream_t)stream));
}
