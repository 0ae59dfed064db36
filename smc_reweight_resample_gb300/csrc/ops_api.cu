// ops_api.cu -- C ABI of beam selection, state and page housekeeping and the distillation loss: host-side argument checks
// and launches.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "ops_launch.cuh"
#include "smcsd.h"
#include "smcsd_launch.cuh"

using namespace smcsd;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? SMCSD_OK : SMCSD_ERR_CUDA; }
int elem_bytes(int dtype) { return dtype == SMCSD_F32 ? 4 : 2; }
bool finite_pos(float v) { return v > 0.0f && isfinite(v); }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) return SMCSD_ERR_INVALID_ARG;
    if (((uintptr_t)ws & 255u) != 0 || ws_bytes < need) return SMCSD_ERR_WORKSPACE;
    return SMCSD_OK;
}

// Memory that a call reads or writes, and whether what it writes meets what it reads, which other blocks may not have read yet.
struct Span {
    const void* at;
    unsigned __int128 bytes;
    Span(const void* p, long long n, long long each) : at(p), bytes((unsigned __int128)n * (unsigned long long)each) {}
};
bool meet(const Span& a, const Span& b) {
    const unsigned __int128 x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}
bool meet(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span& a : written)
        for (const Span& b : read)
            if (meet(a, b)) return true;
    return false;
}
// The same of many at once, what is written of what is written too; sorts them.
struct Touched {
    uintptr_t from, to;
    bool written;
};
bool meet(Touched* t, int n) {
    std::sort(t, t + n, [](const Touched& a, const Touched& b) { return a.from < b.from; });
    uintptr_t written = 0, any = 0;  // where what came before ends
    for (int i = 0; i < n; ++i) {
        if (t[i].from < (t[i].written ? any : written)) return true;
        if (t[i].written && t[i].to > written) written = t[i].to;
        if (t[i].to > any) any = t[i].to;
    }
    return false;
}
// The same of two matrices' rows of V elements of e bytes, which may lie between one another.
bool rows_meet(const void* a, long long stride_a, const void* b, long long stride_b, int R, int V, int e) {
    const auto span = [&](const void* p, long long stride) {
        Span s(p, R - 1, stride);
        s.bytes = (s.bytes + (unsigned)V) * (unsigned)e;
        return s;
    };
    if (!meet(span(a, stride_a), span(b, stride_b))) return false;
    if (stride_a != stride_b || R == 1) return true;
    const __int128 s = stride_a, d = (((__int128)(uintptr_t)b - (__int128)(uintptr_t)a) / e % s + s) % s;
    return d < V || s - d < V;
}
// Whether R rows of V elements of e bytes have memory of a span, which may lie between them: rows that begin before its end, and end
// behind its beginning.
bool rows_meet(const void* rows, long long stride, int R, int V, int e, const Span& s) {
    if (!rows || !s.at) return false;
    const auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0 ? 1 : 0); };
    const __int128 step = (__int128)stride * e, from = (__int128)(uintptr_t)s.at - (__int128)(uintptr_t)rows;
    const __int128 first = floor_div(from - (__int128)V * e, step) + 1, last = floor_div(from + (__int128)s.bytes - 1, step);
    return (first > 0 ? first : 0) <= (last < R - 1 ? last : R - 1);
}

// log2 of a page size of 8 .. 256, or -1
int page_shift(int page_size) {
    for (int b = 3; b <= 8; ++b)
        if (page_size == 1 << b) return b;
    return -1;
}

// Tokens, and a row's vectors filled up to whole chunks, are counted in 32 bits.
constexpr int kMostVocab = 0x7fffffff - 65535;

}  // namespace

extern "C" int beam_select(const void* logits, long long row_stride, int dtype, int G, int N, int V, int M, float temperature,
                           const float* scores, const int32_t* finished, int pad_token, int eos_token, int32_t* tokens,
                           int32_t* ancestors, float* out_scores, int32_t* out_finished, void* ws, size_t ws_bytes, void* stream) {
    if (dtype != SMCSD_F32 && dtype != SMCSD_BF16) return SMCSD_ERR_DTYPE;
    if (!logits || !tokens || !ancestors || !out_scores) return SMCSD_ERR_INVALID_ARG;
    if (G <= 0 || N <= 0 || N > kBeamMostBeams || V <= 0 || V > kMostVocab || M <= 0 || M > kBeamMost) return SMCSD_ERR_INVALID_ARG;
    if ((long long)G * N > 0x7fffffffLL || (long long)G * M > 0x7fffffffLL || !finite_pos(temperature) || !isfinite(1.5f / temperature))
        return SMCSD_ERR_INVALID_ARG;
    if (row_stride < V || (uintptr_t)logits % elem_bytes(dtype)) return SMCSD_ERR_INVALID_ARG;
    // outputs that are read while others are written
    if (out_scores == scores || (finished && out_finished == finished)) return SMCSD_ERR_INVALID_ARG;
    if ((long long)N * beam_chunks(V, elem_bytes(dtype)) > kBeamMostChunks) return SMCSD_ERR_INVALID_ARG;
    const BeamLayout L = beam_layout(G * N, V);
    int rc = check_ws(ws, ws_bytes, L.total);
    if (rc) return rc;
    const long long out = (long long)G * M;
    if (meet({{tokens, out, 4}, {ancestors, out, 4}, {out_scores, out, 4}, {out_finished, out, 4}},
             {{scores, (long long)G * N, 4}, {finished, (long long)G * N, 4}}))
        return SMCSD_ERR_INVALID_ARG;
    BeamParams p{};
    p.logits = logits;
    p.row_stride = row_stride;
    p.G = G;
    p.N = N;
    p.V = V;
    p.M = M;
    const double c = 1.0 / (double)temperature;
    p.c_hi = (float)c;
    p.c_lo = (float)(c - (double)p.c_hi);
    p.c2 = (float)(c * 1.4426950408889634074);
    p.scores = scores;
    p.finished = finished;
    p.pad = pad_token;
    p.eos = eos_token;
    p.tokens = tokens;
    p.ancestors = ancestors;
    p.out_scores = out_scores;
    p.out_finished = out_finished;
    p.ws = ws;
    p.maxima = L.maxima;
    p.sums = L.sums;
    p.sets = L.sets;
    p.cpr = beam_chunks(V, elem_bytes(dtype));
    p.div_cpr = make_fastdiv((uint32_t)p.cpr);
    p.T = make_exp2_table();
    return from_cuda(launch_beam(p, dtype, (cudaStream_t)stream));
}

extern "C" int state_reorder(const void* const* src, void* const* dst, const long long* row_bytes, int count,
                             const int32_t* ancestors, int G, int N, int M, void* ws, size_t ws_bytes, void* stream) {
    if (!src || !dst || !row_bytes || !ancestors || count <= 0 || count > kReorderMost) return SMCSD_ERR_INVALID_ARG;
    if (G <= 0 || N <= 0 || M <= 0 || (long long)G * N > 0x7fffffffLL || (long long)G * M > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    const long long most = (long long)G * (N > M ? N : M);  // rows; a tensor has at most 2^46 bytes
    ReorderParams p{};
    Touched t[2 * kReorderMost + 1];
    for (int i = 0; i < count; ++i) {
        if (!src[i] || !dst[i] || row_bytes[i] <= 0 || row_bytes[i] > (1ll << 46) / most) return SMCSD_ERR_INVALID_ARG;
        const uintptr_t a = (uintptr_t)src[i], b = (uintptr_t)dst[i];
        t[2 * i] = Touched{a, a + (uintptr_t)row_bytes[i] * G * N, false};
        t[2 * i + 1] = Touched{b, b + (uintptr_t)row_bytes[i] * G * M, true};
        const uintptr_t all = a | b | (uintptr_t)row_bytes[i];
        p.unit[i] = all % 16 == 0 ? 4 : all % 4 == 0 ? 2 : 0;
        p.src[i] = src[i];
        p.dst[i] = dst[i];
        p.row_units[i] = row_bytes[i] >> p.unit[i];
    }
    // all tensors are moved at one time: a destination may be written before what shares its memory is read, of whichever tensor
    t[2 * count] = Touched{(uintptr_t)ancestors, (uintptr_t)ancestors + 4 * (uintptr_t)((long long)G * M), false};
    if (meet(t, 2 * count + 1)) return SMCSD_ERR_INVALID_ARG;
    p.ancestors = ancestors;
    p.count = count;
    p.G = G;
    p.N = N;
    p.M = M;
    p.ws = ws;
    return from_cuda(launch_reorder(p, (cudaStream_t)stream));
}

static int fork_or_free(const int32_t* parents, const int32_t* lengths, int S, const int32_t* table_in, int32_t* table_out,
                        int pages_per_seq, int page_size, const int32_t* refcount_in, int32_t* refcount_out, int num_pages, void* ws,
                        size_t ws_bytes, void* stream) {
    if (!table_in || !table_out || !refcount_in || !refcount_out) return SMCSD_ERR_INVALID_ARG;
    if (table_in == table_out || refcount_in == refcount_out) return SMCSD_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (S <= 0 || pages_per_seq <= 0 || shift < 0 || num_pages <= 0) return SMCSD_ERR_INVALID_ARG;
    if ((long long)pages_per_seq * page_size > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;
    if ((long long)S * ((pages_per_seq + 1023) / 1024) > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;  // blocks
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    const long long n = (long long)S * pages_per_seq;
    if (meet({{table_out, n, 4}, {refcount_out, num_pages, 4}},
             {{table_in, n, 4}, {refcount_in, num_pages, 4}, {parents, S, 4}, {lengths, S, 4}}))
        return SMCSD_ERR_INVALID_ARG;
    const ForkParams p{parents,  lengths, S,           table_in,  table_out, pages_per_seq,
                       shift,    refcount_in, refcount_out, num_pages, ws};
    return from_cuda(launch_fork(p, (cudaStream_t)stream));
}

extern "C" int kv_fork(const int32_t* parents, const int32_t* lengths, int S, const int32_t* table_in, int32_t* table_out,
                       int pages_per_seq, int page_size, const int32_t* refcount_in, int32_t* refcount_out, int num_pages, void* ws,
                       size_t ws_bytes, void* stream) {
    if (!parents) return SMCSD_ERR_INVALID_ARG;
    return fork_or_free(parents, lengths, S, table_in, table_out, pages_per_seq, page_size, refcount_in, refcount_out, num_pages, ws,
                        ws_bytes, stream);
}

extern "C" int kv_free(const int32_t* lengths, int S, const int32_t* table_in, int32_t* table_out, int pages_per_seq, int page_size,
                       const int32_t* refcount_in, int32_t* refcount_out, int num_pages, void* ws, size_t ws_bytes, void* stream) {
    if (!lengths) return SMCSD_ERR_INVALID_ARG;
    return fork_or_free(nullptr, lengths, S, table_in, table_out, pages_per_seq, page_size, refcount_in, refcount_out, num_pages, ws,
                        ws_bytes, stream);
}

extern "C" int kv_compact(int S, const int32_t* table_in, int32_t* table_out, int pages_per_seq, const int32_t* refcount_in,
                          int32_t* refcount_out, int num_pages, int32_t* src, int32_t* dst, int32_t* counts, void* ws, size_t ws_bytes,
                          void* stream) {
    if (!table_in || !table_out || !refcount_in || !refcount_out || !counts) return SMCSD_ERR_INVALID_ARG;
    if (table_in == table_out || refcount_in == refcount_out) return SMCSD_ERR_INVALID_ARG;
    if (S <= 0 || pages_per_seq <= 0 || num_pages <= 0 || num_pages > kMostVocab) return SMCSD_ERR_INVALID_ARG;
    if (num_pages > 1 && (!src || !dst || src == dst)) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, compact_bytes(num_pages));
    if (rc) return rc;
    const long long n = (long long)S * pages_per_seq;
    if (meet({{table_out, n, 4}, {refcount_out, num_pages, 4}, {src, num_pages / 2, 4}, {dst, num_pages / 2, 4}, {counts, 2, 4}},
             {{table_in, n, 4}, {refcount_in, num_pages, 4}}))
        return SMCSD_ERR_INVALID_ARG;
    // the moves and their number are read again once the table and the counts are written
    const auto out = [](const void* at, long long words) { return Touched{(uintptr_t)at, (uintptr_t)at + 4 * (uintptr_t)words, at && words > 0}; };
    Touched outs[] = {out(table_out, n), out(refcount_out, num_pages), out(src, num_pages / 2), out(dst, num_pages / 2), out(counts, 2)};
    if (meet(outs, 5)) return SMCSD_ERR_INVALID_ARG;
    CompactParams p{};
    p.table_in = table_in;
    p.table_out = table_out;
    p.entries = (long long)S * pages_per_seq;
    p.ref_in = refcount_in;
    p.ref_out = refcount_out;
    p.num_pages = num_pages;
    p.src = src;
    p.dst = dst;
    p.counts = counts;
    p.ws = ws;
    p.place = compact_place();
    return from_cuda(launch_compact(p, (cudaStream_t)stream));
}

extern "C" int kv_copy_pages(void* const* caches, int n_caches, long long page_bytes, int num_pages, const int32_t* src,
                             const int32_t* dst, int n, const int32_t* count, void* ws, size_t ws_bytes, void* stream) {
    if (!caches || n_caches <= 0 || n_caches > kCopyMost || !src || !dst) return SMCSD_ERR_INVALID_ARG;
    if (page_bytes <= 0 || page_bytes % 16 || page_bytes > (1ll << 32) || num_pages <= 0 || n <= 0) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    CopyParams p{};
    for (int i = 0; i < n_caches; ++i) {
        if (!caches[i] || !aligned16(caches[i])) return SMCSD_ERR_INVALID_ARG;
        p.cache[i] = caches[i];
    }
    p.caches = n_caches;
    p.page_vecs = page_bytes / 16;
    p.src = src;
    p.dst = dst;
    p.n = n;
    p.count = count;
    p.num_pages = num_pages;
    p.ws = ws;
    return from_cuda(launch_copy_pages(p, (cudaStream_t)stream));
}

extern "C" int distill_loss(const void* logits, long long row_stride, int dtype, int R, int V, const int32_t* top_tokens,
                            const float* top_values, int K, float temperature, int rest, const float* weight, float* loss, void* dlogits,
                            long long dlogits_stride, void* ws, size_t ws_bytes, void* stream) {
    if (dtype != SMCSD_F32 && dtype != SMCSD_BF16) return SMCSD_ERR_DTYPE;
    if (!logits || !top_tokens || !top_values || (!loss && !dlogits)) return SMCSD_ERR_INVALID_ARG;
    if (R <= 0 || V <= 0 || K <= 0 || K > kDistillMostTokens || !finite_pos(temperature) || !isfinite(1.5f / temperature))
        return SMCSD_ERR_INVALID_ARG;
    const int b = elem_bytes(dtype);
    if ((long long)V * b > kDistillMostCtas * kDistillMostBytes - 32) return SMCSD_ERR_INVALID_ARG;
    if (row_stride < V || (dlogits && dlogits_stride < V) || (rest != 0 && rest != 1)) return SMCSD_ERR_INVALID_ARG;
    if ((uintptr_t)logits % b || (uintptr_t)dlogits % b || (long long)R * kDistillMostCtas > 0x7fffffffLL) return SMCSD_ERR_INVALID_ARG;
    // in place: every element is written by the block that has read it, where both rows are the same memory
    if (dlogits == logits && dlogits_stride != row_stride) return SMCSD_ERR_INVALID_ARG;
    int rc = check_ws(ws, ws_bytes, 256);
    if (rc) return rc;
    if (dlogits && dlogits != logits && rows_meet(logits, row_stride, dlogits, dlogits_stride, R, V, b)) return SMCSD_ERR_INVALID_ARG;
    const Span out(loss, R, 4), lists[] = {{top_tokens, (long long)R * K, 4}, {top_values, (long long)R * K, 4}, {weight, R, 4}};
    if (rows_meet(logits, row_stride, R, V, b, out) || rows_meet(dlogits, dlogits_stride, R, V, b, out)) return SMCSD_ERR_INVALID_ARG;
    for (const Span& list : lists)
        if (meet(out, list) || rows_meet(dlogits, dlogits_stride, R, V, b, list)) return SMCSD_ERR_INVALID_ARG;
    DistillParams p{};
    p.logits = logits;
    p.row_stride = row_stride;
    p.R = R;
    p.V = V;
    p.K = K;
    p.tokens = top_tokens;
    p.values = top_values;
    p.c = 1.0f / temperature;
    p.c2 = (float)(1.4426950408889634074 / (double)temperature);
    p.rest = rest != 0;
    p.weight = weight;
    p.loss = loss;
    p.grad = dlogits;
    p.grad_stride = dlogits_stride;
    p.ws = ws;
    return from_cuda(launch_distill(p, dtype, (cudaStream_t)stream));
}
