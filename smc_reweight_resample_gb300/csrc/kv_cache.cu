// kv_cache.cu -- page tables and slots of a step's new tokens, and their keys and values' way into
// the paged cache.
#include <cooperative_groups.h>

#include "serve_launch.cuh"
#include "smcsd_launch.cuh"

namespace cg = cooperative_groups;

namespace smcsd {

// ------------------------------------------------------------------------------------------
// kv_slot_map
// ------------------------------------------------------------------------------------------

constexpr int kSlotThreads = 1024;
constexpr int kSlotWarps = kSlotThreads / 32;

struct SlotSeq {
    int first, n;      // rows
    int ctx;
    int j0, j1;        // written pages
    bool ok;
};

__device__ __forceinline__ SlotSeq slot_seq(const SlotParams& p, int s) {
    SlotSeq q;
    q.n = nodes_of(p.n, s, q.first, p.ws);
    q.ctx = __ldg(p.ctx_len + s);
    q.ok = q.ctx >= 0 && (long long)q.ctx + q.n <= ((long long)p.pages_per_seq << p.page_shift);
    if (!q.ok) raise_error(p.ws, kErrRange);
    q.j0 = q.ok ? q.ctx >> p.page_shift : 0;
    q.j1 = q.ok && q.n > 0 ? (q.ctx + q.n + p.page_size - 1) >> p.page_shift : q.j0;
    return q;
}

// Whether a written table entry needs a page: 0 no, 1 empty, 2 shared.
__device__ __forceinline__ int slot_need(const SlotParams& p, int id) {
    if (id == -1) return 1;
    if (id < 0 || id >= p.num_pages) {
        raise_error(p.ws, kErrRange);
        return 0;
    }
    const int ref = __ldg(p.ref_in + id);
    if (ref < 1) raise_error(p.ws, kErrRange);  // held and free at once
    return ref > 1 ? 2 : 0;
}

// Exclusive prefix over the block's warps of one value per warp (lane 0's), and the total.
__device__ __forceinline__ int warp_prefix(int v, int* s, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    int x = s[lane], in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += t;
    }
    total = __shfl_sync(0xffffffffu, in, 31);
    const int before = __shfl_sync(0xffffffffu, in - x, warp);
    __syncthreads();
    return before;
}

// One cluster. Its warps share out the sequences and the pages, both in order: a warp takes a run of
// sequences (their demand) and a run of pages (how many are free). The counts meet in the cluster's
// shared memories; then every free page knows its place in the list of free pages and every sequence
// the place where its pages begin, so the k-th page needed gets the k-th free page whatever runs first. Latency bounds it: 7.2 us
// for 16 sequences of one token (one block: its launch and three dependent loads on either side of a barrier), 10.8 us for 256 of
// nine after a resampling (eight blocks: two barriers of the cluster, and a sequence and some runs of pages for each warp in turn),
// whose bytes would take 0.2 us.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const __grid_constant__ SlotParams p) {
    __shared__ int s_warp[kSlotWarps];
    __shared__ int s_tot[2];
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gw = rank * kSlotWarps + warp, nw = C * kSlotWarps;
    int32_t* free_list = ws_ptr<int32_t>(p.ws, p.free_list);
    int32_t* demand = ws_ptr<int32_t>(p.ws, p.demand);
    const int S = p.n.S;
    // sequences of this warp
    const int sper = (S + nw - 1) / nw, s0 = min(S, gw * sper), s1 = min(S, s0 + sper);
    int want = 0;
    for (int s = s0; s < s1; ++s) {
        const SlotSeq q = slot_seq(p, s);
        const int32_t* row = p.table_in + (long long)s * p.pages_per_seq;
        int d = 0;
        for (int j = q.j0; j < q.j1; j += 32) {
            const bool need = j + lane < q.j1 && slot_need(p, __ldg(row + j + lane)) != 0;
            d += __popc(__ballot_sync(0xffffffffu, need));
        }
        if (lane == 0) demand[s] = d;
        want += d;
    }
    // ragged rows that no sequence has, or whose sequence is refused, keep this; the others are written behind the barriers
    if (p.n.offsets)
        for (long long i = (long long)rank * kSlotThreads + threadIdx.x; i < p.n.R; i += (long long)C * kSlotThreads) p.slots[i] = -1;
    // pages of this warp, in runs of 32 that a ballot counts
    const int runs = (p.num_pages + 31) / 32, rper = (runs + nw - 1) / nw;
    const int r0 = min(runs, gw * rper), r1 = min(runs, r0 + rper);
    int have = 0;
    for (int r = r0; r < r1; ++r) {
        const int id = r * 32 + lane;
        have += __popc(__ballot_sync(0xffffffffu, id < p.num_pages && __ldg(p.ref_in + id) == 0));
    }
    int want_block, have_block;
    int want_at = warp_prefix(want, s_warp, want_block);
    int have_at = warp_prefix(have, s_warp, have_block);
    if (threadIdx.x == 0) {
        s_tot[0] = want_block;
        s_tot[1] = have_block;
    }
    cl.sync();
    int want_all = 0, have_all = 0;
    for (int c = 0; c < C; ++c) {
        const int* t = cl.map_shared_rank(s_tot, c);
        const int w = t[0], h = t[1];
        if (c < rank) want_at += w, have_at += h;
        want_all += w;
        have_all += h;
    }
    for (int r = r0; r < r1; ++r) {
        const int id = r * 32 + lane;
        const int ref = id < p.num_pages ? __ldg(p.ref_in + id) : 1;
        const unsigned b = __ballot_sync(0xffffffffu, ref == 0);
        const int k = have_at + __popc(b & ((1u << lane) - 1u));
        const bool taken = ref == 0 && k < want_all;
        if (taken) free_list[k] = id;
        if (id < p.num_pages) p.ref_out[id] = taken ? 1 : ref;
        have_at += __popc(b);
    }
    cl.sync();  // the list and the counts are there; no block's shared memory is read any more
    for (int s = s0; s < s1; ++s) {
        const SlotSeq q = slot_seq(p, s);
        const int32_t* row = p.table_in + (long long)s * p.pages_per_seq;
        int32_t* to = p.table_out + (long long)s * p.pages_per_seq;
        int at = want_at, src = -1, dst = -1;
        for (int j0 = 0; j0 < p.pages_per_seq; j0 += 32) {
            const int j = j0 + lane;
            const bool in = j < p.pages_per_seq;
            int id = in ? __ldg(row + j) : -1;
            const bool written = in && j >= q.j0 && j < q.j1;
            const int need = written ? slot_need(p, id) : 0;
            const unsigned b = __ballot_sync(0xffffffffu, need != 0);
            if (need) {
                const int k = at + __popc(b & ((1u << lane) - 1u));
                int got = -1;
                if (k < have_all)
                    got = __ldcg(free_list + k);
                else
                    raise_error(p.ws, kErrPages);
                if (need == 2) {
                    atomicSub(p.ref_out + id, 1);
                    if (j == q.j0 && (q.ctx & (p.page_size - 1))) src = id, dst = got;
                }
                id = got;
            }
            at += __popc(b);
            if (in) to[j] = id;
        }
        want_at += demand[s];
        if (src >= 0) {  // one lane at most: the first written page's
            p.copy_src[s] = dst >= 0 ? src : -1;
            p.copy_dst[s] = dst;
        }
        const unsigned any = __ballot_sync(0xffffffffu, src >= 0);
        if (!any && lane == 0) p.copy_src[s] = p.copy_dst[s] = -1;
        __syncwarp();
        for (int i = lane; i < q.n; i += 32) {
            int64_t slot = -1;
            if (q.ok) {
                const int pos = q.ctx + i, id = to[pos >> p.page_shift];
                if (id >= 0 && id < p.num_pages) slot = ((int64_t)id << p.page_shift) + (pos & (p.page_size - 1));
            }
            p.slots[q.first + i] = slot;
        }
    }
}

cudaError_t launch_slot_map(const SlotParams& p, cudaStream_t st) {
    // a warp reads 32 pages at a time: one block for up to 4096 pages or 32 sequences, then as many
    // blocks as leave every warp about 128 pages and one sequence, at most a portable cluster of 8
    int C = 1;
    while (C < 8 && (p.num_pages > C * kSlotWarps * 128 || p.n.S > C * kSlotWarps)) C *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kSlotThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, slot_map_kernel, p);
}

// ------------------------------------------------------------------------------------------
// kv_append
// ------------------------------------------------------------------------------------------

constexpr int kAppendThreads = 256;

// Blocks below `writers` write new tokens, one 16-byte vector of the key and of the value per thread;
// each block after them copies one sequence's shared page. The two touch different slots. One load and one store a
// thread: 3.9 us for 128 sequences of five tokens with their copies (13 MB, latency), 31.8 us for prompts of 25000 tokens (204 MB,
// 6.4 TB/s, 96 % of a copy's rate: memory).
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p, int writers) {
    const uint4* kn = static_cast<const uint4*>(p.k_new);
    const uint4* vn = static_cast<const uint4*>(p.v_new);
    uint4* kc = static_cast<uint4*>(p.k_cache);
    uint4* vc = static_cast<uint4*>(p.v_cache);
    const int rv = p.row_vecs, hv = p.Hkv * rv;
    if ((int)blockIdx.x < writers) {
        const long long n = (long long)p.R * hv;
        for (long long i = (long long)blockIdx.x * kAppendThreads + threadIdx.x; i < n;
             i += (long long)writers * kAppendThreads) {
            const int r = (int)(i / hv), e = (int)(i - (long long)r * hv);
            const int64_t slot = __ldg(p.slots + r);
            if (slot < 0) continue;
            const int64_t page = slot >> p.page_shift;
            if (page >= p.num_pages) {
                raise_error(p.ws, kErrRange);
                continue;
            }
            const int h = e / rv, v = e - h * rv;
            const long long from = (long long)r * p.token_vecs + e;
            const long long to = ((page * p.Hkv + h) * p.page_size + (slot & (p.page_size - 1))) * rv + v;
            const uint4 a = __ldg(kn + from), b = __ldg(vn + from);
            kc[to] = a;
            vc[to] = b;
        }
        return;
    }
    const int s = blockIdx.x - writers;
    const int src = __ldg(p.copy_src + s), dst = __ldg(p.copy_dst + s);
    if (src < 0) return;
    const int c = __ldg(p.ctx_len + s);
    if (src >= p.num_pages || dst < 0 || dst >= p.num_pages || c < 0) {
        if (threadIdx.x == 0) raise_error(p.ws, kErrRange);
        return;
    }
    const int part = (c & (p.page_size - 1)) * rv;  // vectors of each head
    const int head = p.page_size * rv;
    for (int i = threadIdx.x; i < part * p.Hkv; i += kAppendThreads) {
        const int h = i / part, e = i - h * part;
        const long long from = ((long long)src * p.Hkv + h) * head + e, to = ((long long)dst * p.Hkv + h) * head + e;
        const uint4 a = kc[from], b = vc[from];
        kc[to] = a;
        vc[to] = b;
    }
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
    const long long n = (long long)p.R * p.Hkv * p.row_vecs;
    long long writers = (n + kAppendThreads - 1) / kAppendThreads;
    const long long cap = (long long)device_sm_count() * 32;
    if (writers > cap) writers = cap;
    const int copies = p.copy_src ? p.S : 0;
    append_kernel<<<(unsigned)(writers + copies), kAppendThreads, 0, st>>>(p, (int)writers);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------------
// tree_mask
// ------------------------------------------------------------------------------------------

constexpr int kMaskThreads = 128;
constexpr int kMaskShared = 4096;  // parents of longer sequences are read through L1

// One block per sequence, one thread per node: the walk from a node to its root meets falling
// indices, so the words of its row are finished from the last to the first. The walk's chain of loads bounds it: 3.1 us for
// 8 trees of 64 nodes, 34 us for 8 of 512.
__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const __grid_constant__ MaskParams p) {
    __shared__ int s_parent[kMaskShared];
    const int s = blockIdx.x;
    int first;
    const int n = nodes_of(p.n, s, first, p.ws);
    for (int i = threadIdx.x; i < min(n, kMaskShared); i += kMaskThreads) s_parent[i] = __ldg(p.parents + first + i);
    __syncthreads();
    for (int t = threadIdx.x; t < n; t += kMaskThreads) {
        uint32_t* row = p.mask + (long long)(first + t) * p.words;
        int at = t;
        for (int w = p.words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            while (at >= 0 && (at >> 5) == w) {
                bits |= 1u << (at & 31);
                const int up = at < kMaskShared ? s_parent[at] : __ldg(p.parents + first + at);
                if (up < -1 || up >= at) {
                    raise_error(p.ws, kErrRange);
                    at = -1;
                } else {
                    at = up;
                }
            }
            row[w] = bits;
        }
    }
}

cudaError_t launch_tree_mask(const MaskParams& p, cudaStream_t st) {
    tree_mask_kernel<<<p.n.S, kMaskThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace smcsd
