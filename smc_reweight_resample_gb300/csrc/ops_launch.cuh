// ops_launch.cuh -- launch parameters of beam selection, of the page housekeeping and of the distillation loss.
#pragma once

#include "smcsd_internal.cuh"

namespace smcsd {

// ------------------------------------------------------------------------------------------
// beam selection
// ------------------------------------------------------------------------------------------

constexpr int kBeamMostBeams = 256;  // of a group
constexpr int kBeamMost = 256;       // selected of a group
constexpr int kBeamSets = 16;        // sets of 16 16-byte vectors in a chunk of 4 KB
constexpr int kBeamMostChunks = 40960;  // of a group: their scores stand in shared memory

struct BeamParams {
    const void* logits;
    long long row_stride;  // elements
    int G, N, V, M;
    float c_hi, c_lo, c2;  // c = 1 / temperature as a double-float; c log2(e)
    const float* scores;
    const int32_t* finished;
    int pad, eos;
    int32_t* tokens;
    int32_t* ancestors;
    float* out_scores;
    int32_t* out_finished;
    void* ws;
    size_t maxima; // float [G * N, cpr]             of a chunk
    size_t sums;   // float [G * N, cpr]             relative to it
    size_t sets;   // float [G * N, cpr, kBeamSets]  maximum of a set
    int cpr, blocks;  // chunks of a row, blocks of a group
    FastDiv div_cpr;
    Exp2Table T;
};

// Chunks of a row that may begin anywhere in its first 16-byte vector.
inline int beam_chunks(int V, int bytes) { return (int)(((long long)V * bytes + 15 + kChunkBytes - 1) / kChunkBytes); }

struct BeamLayout {
    size_t maxima, sums, sets, total;
};
inline BeamLayout beam_layout(int rows, int V) {
    const size_t n = (size_t)rows * (size_t)beam_chunks(V, 4);
    BeamLayout L{};
    size_t o = kFrontBytes;
    L.maxima = o;
    o = align256(o + 4 * n);
    L.sums = o;
    o = align256(o + 4 * n);
    L.sets = o;
    o = align256(o + 4 * kBeamSets * n);
    L.total = o;
    return L;
}

cudaError_t launch_beam(const BeamParams& p, int dtype, cudaStream_t st);

// ------------------------------------------------------------------------------------------
// states and pages
// ------------------------------------------------------------------------------------------

constexpr int kReorderMost = 64;  // tensors of a call

struct ReorderParams {
    const void* src[kReorderMost];
    void* dst[kReorderMost];
    long long row_units[kReorderMost];  // of `unit` bytes
    unsigned char unit[kReorderMost];   // log2: 0, 2 or 4
    unsigned first[kReorderMost + 1];   // first block
    const int32_t* ancestors;
    int count, G, N, M;
    void* ws;
};

struct ForkParams {
    const int32_t* parents;
    const int32_t* lengths;
    int S;
    const int32_t* table_in;
    int32_t* table_out;
    int pages_per_seq, page_shift;
    const int32_t* ref_in;
    int32_t* ref_out;
    int num_pages;
    void* ws;
};

struct CompactParams {
    const int32_t* table_in;
    int32_t* table_out;
    long long entries;
    const int32_t* ref_in;
    int32_t* ref_out;
    int num_pages;
    int32_t* src;
    int32_t* dst;
    int32_t* counts;  // moves, pages in use
    void* ws;
    size_t place;  // int32 [num_pages]: which move a page from behind is
    bool small;
};

inline size_t compact_place() { return kFrontBytes; }
inline size_t compact_bytes(int num_pages) { return align256(compact_place() + 4 * (size_t)num_pages); }

constexpr int kCopyMost = 256;  // caches of a call

struct CopyParams {
    void* cache[kCopyMost];
    int caches;
    long long page_vecs;  // 16-byte vectors of a page
    const int32_t* src;
    const int32_t* dst;
    int n;
    const int32_t* count;
    int num_pages;
    void* ws;
};

cudaError_t launch_reorder(const ReorderParams& p, cudaStream_t st);
cudaError_t launch_fork(const ForkParams& p, cudaStream_t st);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t st);
cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t st);

// ------------------------------------------------------------------------------------------
// distillation loss
// ------------------------------------------------------------------------------------------

constexpr int kDistillMostTokens = 256;              // of a row's list
constexpr int kDistillMostCtas = 16;                 // of a row
constexpr long long kDistillMostBytes = 100 * 1024;  // of a row in one block's shared memory

struct DistillParams {
    const void* logits;
    long long row_stride;
    int R, V, K;
    const int32_t* tokens;
    const float* values;
    float c, c2;  // 1 / temperature; that times log2(e)
    bool rest;
    const float* weight;
    float* loss;
    void* grad;
    long long grad_stride;
    void* ws;
    int ctas, vecs;  // of a row; 16-byte vectors of a block's share
};

cudaError_t launch_distill(const DistillParams& p, int dtype, cudaStream_t st);

}  // namespace smcsd
