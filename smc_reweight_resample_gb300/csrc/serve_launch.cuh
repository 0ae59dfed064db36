// serve_launch.cuh -- launch parameters of the page-table, cache-write, node-mask and logits kernels.
#pragma once

#include "smcsd_internal.cuh"

namespace smcsd {

// The nodes of every sequence: rows s*T .. s*T+T-1, or given by offsets.
struct Nodes {
    const int32_t* offsets;
    int S, T, R;
};

// First row and number of nodes of sequence s; none (and an error) if the offsets do not fit.
__device__ __forceinline__ int nodes_of(const Nodes& n, int s, int& first, void* ws) {
    if (!n.offsets) {
        first = s * n.T;
        return n.T;
    }
    const int a = __ldg(n.offsets + s), b = __ldg(n.offsets + s + 1);
    first = a;
    if (a < 0 || b < a || b > n.R || b - a > n.T) {
        raise_error(ws, kErrRange);
        return 0;
    }
    return b - a;
}

struct SlotParams {
    const int32_t* ctx_len;
    Nodes n;
    const int32_t* table_in;
    int32_t* table_out;
    int pages_per_seq, page_size, page_shift;
    const int32_t* ref_in;
    int32_t* ref_out;
    int num_pages;
    int64_t* slots;
    int32_t* copy_src;
    int32_t* copy_dst;
    void* ws;
    size_t free_list;  // int32 [num_pages]: free pages in ascending order
    size_t demand;     // int32 [S]: pages that a sequence takes
};

struct AppendParams {
    const void* k_new;
    const void* v_new;
    long long token_vecs;  // 16-byte vectors from one token to the next
    int R, Hkv, row_vecs;  // vectors in one head's row
    const int64_t* slots;
    const int32_t* copy_src;
    const int32_t* copy_dst;
    const int32_t* ctx_len;
    int S;
    void* k_cache;
    void* v_cache;
    int page_size, page_shift, num_pages;
    void* ws;
};

struct MaskParams {
    const int32_t* parents;
    Nodes n;
    uint32_t* mask;
    int words;
    void* ws;
};

struct LogitsParams {
    const void* logits;
    void* out;
    Nodes n;
    int V;
    bool vec;  // 16-byte aligned rows
    const int32_t* node_tokens;
    const uint32_t* mask;
    int words;
    const int32_t* hist_tokens;
    const int32_t* hist_offsets;
    int n_hist, n_bias;
    const float* repetition;
    const float* presence;
    const float* frequency;
    const int32_t* bias_tokens;
    const float* bias_values;
    const int32_t* bias_offsets;
    const uint32_t* allowed;
    int allowed_words;
    void* ws;
};

inline size_t slot_map_free_list() { return kFrontBytes; }
inline size_t slot_map_demand(int num_pages) { return align256(slot_map_free_list() + 4 * (size_t)num_pages); }
inline size_t slot_map_bytes(int S, int num_pages) { return align256(slot_map_demand(num_pages) + 4 * (size_t)S); }

cudaError_t launch_slot_map(const SlotParams& p, cudaStream_t st);
cudaError_t launch_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_tree_mask(const MaskParams& p, cudaStream_t st);
cudaError_t launch_logits(const LogitsParams& p, int dtype, cudaStream_t st);

}  // namespace smcsd
