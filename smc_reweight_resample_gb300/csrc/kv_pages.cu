// kv_pages.cu -- sequences' states and pages: rows of states by ancestors, tables forked and freed, pages in use moved to the
// front of the cache, pages copied.
#include <cooperative_groups.h>

#include "ops_launch.cuh"
#include "smcsd_launch.cuh"

namespace cg = cooperative_groups;

namespace smcsd {

// ------------------------------------------------------------------------------------------
// state_reorder
// ------------------------------------------------------------------------------------------

constexpr int kReorderThreads = 256;
constexpr int kReorderUnits = 4;  // units of a thread and turn
constexpr long long kReorderTurn = kReorderThreads * kReorderUnits;

template <typename U>
__device__ __forceinline__ void reorder_units(const ReorderParams& p, const int32_t* ancestors, int t, int block, int blocks) {
    const U* src = static_cast<const U*>(p.src[t]);
    U* dst = static_cast<U*>(p.dst[t]);
    const long long w = p.row_units[t], n = w * p.G * p.M;
    for (long long i0 = block * kReorderTurn + threadIdx.x; i0 < n; i0 += blocks * kReorderTurn) {
        U x[kReorderUnits];
        bool there[kReorderUnits];
#pragma unroll
        for (int k = 0; k < kReorderUnits; ++k) {
            const long long i = i0 + k * kReorderThreads;
            there[k] = i < n;
            if (there[k]) {
                const int row = (int)(i / w), g = row / p.M, a = __ldg(ancestors + row);
                there[k] = a >= 0 && a < p.N;
                if (there[k])
                    x[k] = src[((long long)g * p.N + a) * w + (i - row * w)];
                else
                    raise_error(p.ws, kErrRange);
            }
        }
#pragma unroll
        for (int k = 0; k < kReorderUnits; ++k)
            if (there[k]) dst[i0 + k * kReorderThreads] = x[k];
    }
}

// All tensors in one launch: each has a run of blocks. 2.7 us for 128 rows of 12 KB in three tensors (1.6 MB either way): the launch, and
// two loads one after the other.
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int32_t* ancestors = after_wait(p.ancestors);
    int t = 0;
    while (blockIdx.x >= p.first[t + 1]) ++t;
    const int block = (int)(blockIdx.x - p.first[t]), blocks = (int)(p.first[t + 1] - p.first[t]);
    if (p.unit[t] == 4)
        reorder_units<uint4>(p, ancestors, t, block, blocks);
    else if (p.unit[t] == 2)
        reorder_units<uint32_t>(p, ancestors, t, block, blocks);
    else
        reorder_units<unsigned char>(p, ancestors, t, block, blocks);
}

cudaError_t launch_reorder(const ReorderParams& p0, cudaStream_t st) {
    ReorderParams p = p0;
    const long long cap = 16ll * device_sm_count();  // two waves of eight blocks an SM
    for (int t = 0; t < p.count; ++t) {
        const long long n = p.row_units[t] * p.G * p.M;
        long long blocks = (n + kReorderTurn - 1) / kReorderTurn;
        if (blocks > cap) blocks = cap;
        p.first[t + 1] = p.first[t] + (unsigned)blocks;
    }
    return launch_waiting(reorder_kernel, dim3(p.first[p.count]), kReorderThreads, 0, 0, st, p);
}

// ------------------------------------------------------------------------------------------
// kv_fork, kv_free
// ------------------------------------------------------------------------------------------

constexpr int kForkThreads = 512;  // at most
constexpr int kForkEntries = 4;   // of a thread
constexpr int kForkCounts = 8;    // of a thread
// Entries and pages that one cluster takes. Us by it / by two launches, as many pages as entries, forked: 2064 2.6 / 3.0, 4096 2.7 / 3.7,
// 8192 4.0 / 3.9, 16384 6.4 / 3.9, 49152 15.8 / 4.3; freed: 2064 2.5 / 2.4, 4096 2.6 / 2.6, 8192 3.8 / 2.7, 16384 6.2 / 2.8. Two launches take 2
// us more to issue where the host is behind.
constexpr int kForkMost = 8192;

// A page id of a table: whether it is counted. -1 is no page.
__device__ __forceinline__ bool fork_counts(const ForkParams& p, int id) {
    if (id >= 0 && id < p.num_pages) return true;
    if (id != -1) raise_error(p.ws, kErrRange);
    return false;
}

// Sequence s's parent, and how many entries of the parent's row it takes.
__device__ __forceinline__ void fork_row(const ForkParams& p, int s, int& parent, int& pages) {
    parent = p.parents ? __ldg(p.parents + s) : s;
    const int length = p.lengths ? __ldg(p.lengths + s) : INT_MAX;
    pages = length == INT_MAX ? p.pages_per_seq : (int)(((long long)length + (1 << p.page_shift) - 1) >> p.page_shift);
    if (parent < -1 || parent >= p.S || length < 0) {
        raise_error(p.ws, kErrRange);  // kept as it is
        parent = s;
        pages = p.pages_per_seq;
    }
    if (parent < 0) pages = 0;
}
// Counts change where an entry does: what a sequence keeps costs no atomic.
__device__ __forceinline__ void fork_change(const ForkParams& p, int id, int old) {
    if (fork_counts(p, id)) atomicAdd(p.ref_out + id, 1);
    if (fork_counts(p, old) && atomicSub(p.ref_out + old, 1) <= 0) raise_error(p.ws, kErrRange);  // held, but not counted
}

// Small tables: one cluster copies the counts and writes the new table, meets, and changes the counts. 2.5 to 2.8 us for 16 sequences of 129
// pages and 2128 counts: latency.
constexpr int kForkClusterThreads = 512;
__global__ void __launch_bounds__(kForkClusterThreads) fork_small_kernel(const __grid_constant__ ForkParams p0, const FastDiv by_row) {
    griddep_wait();
    griddep_launch_dependents();
    ForkParams p = p0;
    p.parents = after_wait(p0.parents);
    p.lengths = after_wait(p0.lengths);
    p.table_in = after_wait(p0.table_in);
    p.ref_in = after_wait(p0.ref_in);
    cg::cluster_group cl = cg::this_cluster();
    const int first = (int)cl.block_rank() * kForkClusterThreads + threadIdx.x, step = (int)cl.num_blocks() * kForkClusterThreads;
    const int P = p.pages_per_seq, n = p.S * P;
#pragma unroll 4
    for (int i = first; i < p.num_pages; i += step) p.ref_out[i] = __ldg(p.ref_in + i);
    for (int i = first; i < n; i += step) {
        const int s = (int)fast_div((uint32_t)i, by_row), j = i - s * P;
        int parent, pages;
        fork_row(p, s, parent, pages);
        p.table_out[i] = j < pages ? __ldg(p.table_in + parent * P + j) : -1;
    }
    cl.sync();
    for (int i = first; i < n; i += step) {
        const int id = p.table_out[i], old = __ldg(p.table_in + i);  // the thread's own entry
        if (id != old)
            fork_change(p, id, old);
        else
            fork_counts(p, id);
    }
}

__global__ void __launch_bounds__(kForkThreads) fork_counts_kernel(const __grid_constant__ ForkParams p) {
    griddep_wait();
    griddep_launch_dependents();  // the next kernel reads the old table at once
    const int32_t* ref_in = after_wait(p.ref_in);
    const long long i0 = (long long)blockIdx.x * kForkThreads * kForkCounts + threadIdx.x;
    int x[kForkCounts];
#pragma unroll
    for (int k = 0; k < kForkCounts; ++k)
        if (i0 + k * kForkThreads < p.num_pages) x[k] = __ldg(ref_in + i0 + k * kForkThreads);
#pragma unroll
    for (int k = 0; k < kForkCounts; ++k)
        if (i0 + k * kForkThreads < p.num_pages) p.ref_out[i0 + k * kForkThreads] = x[k];
}

// A thread's entries of a row, from `j0`: vectors of four, `step` of them apart, or entries as far apart.
template <bool kWide>
__device__ __forceinline__ unsigned fork_entry(unsigned j0, int k, unsigned step) {
    return kWide ? j0 + (k >> 2) * 4 * step + (k & 3) : j0 + k * step;
}
template <bool kWide>
__device__ __forceinline__ void fork_load(int (&x)[kForkEntries], const int* row, unsigned j0, unsigned step, unsigned P) {
#pragma unroll
    for (int k = 0; k < kForkEntries; k += kWide ? 4 : 1) {
        const unsigned j = fork_entry<kWide>(j0, k, step);
        if (kWide) {
            const int4 v = j < P ? __ldg(reinterpret_cast<const int4*>(row + j)) : make_int4(-1, -1, -1, -1);
            x[k] = v.x, x[k + 1] = v.y, x[k + 2] = v.z, x[k + 3] = v.w;
        } else {
            x[k] = j < P ? __ldg(row + j) : -1;
        }
    }
}

// A block takes entries of one row, four a thread, a row's blocks as many each. Rows of vectors (their length and both tables' addresses
// allow it) in blocks of 256 threads: for 1024 sequences of 2052 pages and 2.1 million counts copied beside them 8.0 us where sequences are
// freed, 195000 entries, and 6.7 where they fork, 176000 (34 MB, 5 us at the copy rate); with 512 threads 0.3 more. Other rows entry by
// entry: 8.9 and 7.6 with 512 threads, 0.7 more with 256. The counts' copies alone take 2.8, the counts that change one by one 1.4 to 2.5.
template <bool kWide>
__global__ void __launch_bounds__(kWide ? kForkThreads / 2 : kForkThreads) fork_kernel(const __grid_constant__ ForkParams p, int pieces) {
    const int s = blockIdx.x / pieces;
    const unsigned P = p.pages_per_seq, step = blockDim.x;
    const unsigned j0 = (blockIdx.x - s * pieces) * step * kForkEntries + (kWide ? 4 : 1) * threadIdx.x;  // may pass 31 bits
    const long long row = (long long)s * P;
    int old[kForkEntries], id[kForkEntries], parent, pages;
    fork_load<kWide>(old, p.table_in + row, j0, step, P);
    fork_row(p, s, parent, pages);
    const unsigned upto = (unsigned)pages < P ? pages : P;
    if (parent != s && upto > 0) fork_load<kWide>(id, p.table_in + (long long)parent * P, j0, step, P);
#pragma unroll
    for (int k = 0; k < kForkEntries; ++k) {
        if (parent == s) id[k] = old[k];
        if (fork_entry<kWide>(j0, k, step) >= upto) id[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kForkEntries; k += kWide ? 4 : 1) {
        const unsigned j = fork_entry<kWide>(j0, k, step);
        if (j >= P) continue;
        if (kWide)
            *reinterpret_cast<int4*>(p.table_out + row + j) = make_int4(id[k], id[k + 1], id[k + 2], id[k + 3]);
        else
            p.table_out[row + j] = id[k];
    }
    griddep_wait();  // the counts have been copied
    griddep_launch_dependents();
#pragma unroll
    for (int k = 0; k < kForkEntries; ++k) {
        if (id[k] != old[k])
            fork_change(p, id[k], old[k]);
        else
            fork_counts(p, id[k]);
    }
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t st) {
    const long long n = (long long)p.S * p.pages_per_seq;
    if (n <= kForkMost && p.num_pages <= kForkMost) {
        // one launch in place of two: two turns of a cluster of eight blocks at most
        const long long most = n > p.num_pages ? n : p.num_pages;
        int C = 1;
        while (C < 8 && most > C * kForkClusterThreads) C *= 2;
        return launch_waiting(fork_small_kernel, dim3(C), kForkClusterThreads, 0, C, st, p, make_fastdiv((uint32_t)p.pages_per_seq));
    }
    const cudaError_t e = launch_waiting(fork_counts_kernel, dim3((unsigned)((p.num_pages - 1) / (kForkThreads * kForkCounts) + 1)), kForkThreads, 0, 0, st, p);
    if (e != cudaSuccess) return e;
    const bool wide = p.pages_per_seq % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.table_in) | reinterpret_cast<uintptr_t>(p.table_out)) & 15u) == 0;
    const int blocks = (p.pages_per_seq - 1) / ((wide ? kForkThreads / 2 : kForkThreads) * kForkEntries) + 1;
    const int per = (p.pages_per_seq - 1) / blocks + 1, threads = (per + 32 * kForkEntries - 1) / (32 * kForkEntries) * 32;
    const int pieces = (p.pages_per_seq - 1) / (threads * kForkEntries) + 1;
    if ((long long)pieces * p.S > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_waiting(wide ? fork_kernel<true> : fork_kernel<false>, dim3((unsigned)pieces * (unsigned)p.S), threads, 0, 0, st, p, pieces);
}

// ------------------------------------------------------------------------------------------
// kv_compact
// ------------------------------------------------------------------------------------------

constexpr int kCompactThreads = 1024;
constexpr int kCompactWarps = kCompactThreads / 32;
constexpr int kCompactMost = 8192;  // table entries that the planning cluster writes

// Table entries and counts of the pages that move, once the moves are known. Counts that another stream changes meanwhile give other
// places at each reading: a place that no move can have is reported and not followed, here and below.
__device__ __forceinline__ void compact_apply(const CompactParams& p, int moves, int used, long long first, long long step) {
    const int32_t* place = ws_ptr<const int32_t>(p.ws, p.place);
    for (long long i = first; i < moves; i += step) {
        const int from = __ldcg(p.src + i), to = __ldcg(p.dst + i);
        if ((unsigned)from < (unsigned)p.num_pages && (unsigned)to < (unsigned)p.num_pages)
            p.ref_out[to] = __ldg(p.ref_in + from);
        else
            raise_error(p.ws, kErrRange);
    }
#pragma unroll 4
    for (long long i = first; i < p.entries; i += step) {
        int id = __ldg(p.table_in + i);
        if (id != -1) {
            if (id < 0 || id >= p.num_pages || __ldg(p.ref_in + id) <= 0)
                raise_error(p.ws, kErrRange);  // left as it is
            else if (id >= used) {
                const int k = __ldcg(place + id);
                if ((unsigned)k < (unsigned)moves)
                    id = __ldcg(p.dst + k);
                else
                    raise_error(p.ws, kErrRange);
            }
        }
        p.table_out[i] = id;
    }
}

// Which page goes where: one cluster. Its warps share out the pages in order, in runs of 32 that a ballot counts. The number
// of pages in use, U, is the border: a hole's place is the number of free pages before it, that of a page from behind the
// number of pages in use between the border and it, so that the k-th page from behind meets the k-th hole whatever runs first.
// 5.6 us for 600 pages and 384 table entries, 9.5 with the table for 16384 and 13824: latency (three meetings of the cluster, two
// passes over a warp's pages).
__global__ void __launch_bounds__(kCompactThreads) compact_plan_kernel(const __grid_constant__ CompactParams p0) {
    griddep_wait();
    griddep_launch_dependents();
    CompactParams p = p0;
    p.ref_in = after_wait(p0.ref_in);
    p.table_in = after_wait(p0.table_in);
    __shared__ int s_warp[kCompactWarps];
    __shared__ int s_tot, s_before;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gw = rank * kCompactWarps + warp, nw = C * kCompactWarps;
    int32_t* place = ws_ptr<int32_t>(p.ws, p.place);
    const int runs = (p.num_pages + 31) / 32, per = (runs + nw - 1) / nw;
    const int r0 = min(runs, gw * per), r1 = min(runs, r0 + per);
    int have = 0;
    for (int r = r0; r < r1; ++r) {
        const int id = r * 32 + lane;
        have += __popc(__ballot_sync(0xffffffffu, id < p.num_pages && __ldg(p.ref_in + id) > 0));
    }
    if (lane == 0) s_warp[warp] = have;
    if (threadIdx.x == 0) s_before = -1;
    __syncthreads();
    int x = s_warp[lane], in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += t;
    }
    int before = __shfl_sync(0xffffffffu, in - x, warp);
    if (threadIdx.x == 31) s_tot = in;
    cl.sync();
    int used = 0;
    for (int c = 0; c < C; ++c) {
        const int t = *cl.map_shared_rank(&s_tot, c);
        if (c < rank) before += t;
        used += t;
    }
    // pages in use before the border, by the warp that the border is in (none's if every page is in use)
    if (used < p.num_pages && used >= r0 * 32 && used < r1 * 32) {
        int n = before;
        for (int r = r0; r <= used / 32; ++r) {
            const int id = r * 32 + lane;
            n += __popc(__ballot_sync(0xffffffffu, id < used && __ldg(p.ref_in + id) > 0));
        }
        if (lane == 0) s_before = n;
    }
    cl.sync();
    int low = used;
    for (int c = 0; c < C; ++c) {
        const int t = *cl.map_shared_rank(&s_before, c);
        if (t >= 0) low = t;
    }
    const int half = p.num_pages / 2, moves = min(max(used - low, 0), half);
    if (gw == 0 && lane == 0) {
        p.counts[0] = moves;
        p.counts[1] = used;
    }
    for (int i = moves + rank * kCompactThreads + threadIdx.x; i < half; i += C * kCompactThreads) p.src[i] = p.dst[i] = -1;
    for (int r = r0; r < r1; ++r) {
        const int id = r * 32 + lane;
        const int ref = id < p.num_pages ? __ldg(p.ref_in + id) : 0;
        const unsigned b = __ballot_sync(0xffffffffu, ref > 0);
        const int held = before + __popc(b & ((1u << lane) - 1u));  // pages in use before this one
        before += __popc(b);
        if (id >= p.num_pages) continue;
        if (ref < 0) raise_error(p.ws, kErrRange);
        if (id < used) {
            if (ref > 0)
                p.ref_out[id] = ref;
            else if ((unsigned)(id - held) < (unsigned)half)
                p.dst[id - held] = id;  // its count comes with its page
        } else {
            p.ref_out[id] = 0;
            if (ref > 0 && (unsigned)(held - low) < (unsigned)half) {
                p.src[held - low] = id;
                place[id] = held - low;
            }
        }
    }
    cl.sync();  // the moves are there; no block's shared memory is read any more
    if (p.small) compact_apply(p, moves, used, rank * kCompactThreads + threadIdx.x, C * kCompactThreads);
}

constexpr int kApplyThreads = 256;

__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(const __grid_constant__ CompactParams p0) {
    griddep_wait();
    griddep_launch_dependents();
    CompactParams p = p0;
    p.ref_in = after_wait(p0.ref_in);
    p.table_in = after_wait(p0.table_in);
    const int moves = min(max(__ldcg(p.counts), 0), p.num_pages / 2);  // the lists' length, whatever has been written there meanwhile
    compact_apply(p, moves, __ldcg(p.counts + 1), (long long)blockIdx.x * kApplyThreads + threadIdx.x,
                  (long long)gridDim.x * kApplyThreads);
}

cudaError_t launch_compact(const CompactParams& p0, cudaStream_t st) {
    CompactParams p = p0;
    p.small = p.entries <= kCompactMost;  // the cluster writes the table too: one launch in place of two
    // as many blocks as leave every warp about 128 pages, at most a portable cluster of 8
    int C = 1;
    while (C < 8 && p.num_pages > C * kCompactWarps * 128) C *= 2;
    const cudaError_t e = launch_waiting(compact_plan_kernel, dim3(C), kCompactThreads, 0, C, st, p);
    if (e != cudaSuccess || p.small) return e;
    const long long cap = 16ll * device_sm_count(), most = p.entries > p.num_pages / 2 ? p.entries : p.num_pages / 2;
    long long b = (most + kApplyThreads - 1) / kApplyThreads;
    return launch_waiting(compact_apply_kernel, dim3((unsigned)(b < cap ? b : cap)), kApplyThreads, 0, 0, st, p);
}

// ------------------------------------------------------------------------------------------
// kv_copy_pages
// ------------------------------------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 8;  // 16-byte vectors of a thread and turn: 32 KB a block

// 115 us for 2800 pages of 32 KB in four caches (734 MB read and written: 6.4 TB/s, 94 % of a copy's rate), 2.2 for 40 of 4 KB.

// An item is one page of one cache; blocks take them in turn.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
    griddep_wait();
    const int32_t *moved = after_wait(p.src), *moved_to = after_wait(p.dst), *count = after_wait(p.count);
    int n = p.n;
    if (count) {
        const int c = __ldg(count);
        if (c < 0 || c > n) {
            if (threadIdx.x == 0) raise_error(p.ws, kErrRange);
            return;
        }
        n = c;
    }
    const long long w = p.page_vecs, pieces = (w + kCopyThreads * kCopyLoads - 1) / (kCopyThreads * kCopyLoads);
    const long long items = (long long)n * p.caches * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long move = it / pieces, piece = it - move * pieces;
        const int i = (int)(move / p.caches), c = (int)(move - (long long)i * p.caches);
        const int src = __ldg(moved + i), dst = __ldg(moved_to + i);
        if (src < 0 && dst < 0) continue;
        if (src < 0 || dst < 0 || src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0) raise_error(p.ws, kErrRange);
            continue;
        }
        const uint4* from = static_cast<const uint4*>(p.cache[c]) + src * w;
        uint4* to = static_cast<uint4*>(p.cache[c]) + dst * w;
        const long long v0 = piece * kCopyThreads * kCopyLoads + threadIdx.x;
        uint4 x[kCopyLoads];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if (v0 + k * kCopyThreads < w) x[k] = from[v0 + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if (v0 + k * kCopyThreads < w) to[v0 + k * kCopyThreads] = x[k];
    }
}

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t st) {
    const long long pieces = (p.page_vecs + kCopyThreads * kCopyLoads - 1) / (kCopyThreads * kCopyLoads);
    const long long items = (long long)p.n * p.caches * pieces, cap = 8ll * device_sm_count();
    return launch_waiting(copy_pages_kernel, dim3((unsigned)(items < cap ? items : cap)), kCopyThreads, 0, 0, st, p);
}

}  // namespace smcsd
