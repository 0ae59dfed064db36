// tree_attention.cu -- attention of drafted tokens over a paged cache: the planning kernel, the
// kernel on the FP32 pipes and the kernel that joins the pieces of a unit (attn_plan.cuh has the cut).
#include "attn_plan.cuh"
#include "smcsd_launch.cuh"

#include <cuda_bf16.h>

namespace smcsd {

// ------------------------------------------------------------------------------------------
// planning: shared tiles of every group, then the items and their places on the line
// ------------------------------------------------------------------------------------------

constexpr int kPlanThreads = 512;

__device__ __forceinline__ void scan_pair(long long& a, long long& b, long long* sa, long long* sb) {
    // exclusive prefix over the block's threads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long va = __shfl_up_sync(0xffffffffu, ia, o), vb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) ia += va, ib += vb;
    }
    if (lane == 31) sa[warp] = ia, sb[warp] = ib;
    __syncthreads();
    if (warp == 0) {
        const int nw = blockDim.x >> 5;
        long long wa = lane < nw ? sa[lane] : 0, wb = lane < nw ? sb[lane] : 0;
        const long long oa = wa, ob = wb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long va = __shfl_up_sync(0xffffffffu, wa, o), vb = __shfl_up_sync(0xffffffffu, wb, o);
            if (lane >= o) wa += va, wb += vb;
        }
        if (lane < nw) sa[lane] = wa - oa, sb[lane] = wb - ob;
        if (lane == 31) sa[32] = wa, sb[32] = wb;
    }
    __syncthreads();
    a = ia - a + sa[warp];
    b = ib - b + sb[warp];
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnParams p) {
    __shared__ int best;
    __shared__ unsigned last;
    __shared__ long long sa[33], sb[33];
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    int* shared = ws_ptr<int>(p.ws, p.L.shared);
    if (p.G > 0) {
        // pages that every sequence of the group has at the same place, all of them full context
        const int s0 = blockIdx.x * p.N;
        if (tid == 0) best = INT_MAX;
        __syncthreads();
        int c = INT_MAX;
        for (int i = tid; i < p.N; i += kPlanThreads) c = min(c, max(0, __ldg(p.ctx_len + s0 + i)));
        if (c != INT_MAX) atomicMin(&best, c);
        __syncthreads();
        const int lim = min(best >> p.page_shift, p.pages_per_seq);
        __syncthreads();
        if (tid == 0) best = lim;
        __syncthreads();
        const int32_t* row = p.table + (long long)s0 * p.pages_per_seq;
        for (long long i = tid; i < (long long)(p.N - 1) * lim; i += kPlanThreads) {
            const int s = (int)(i / lim), j = (int)(i - (long long)s * lim);
            const int id = __ldg(row + j);
            if (id < 0 || id != __ldg(row + (long long)(s + 1) * p.pages_per_seq + j)) atomicMin(&best, j);
        }
        __syncthreads();
        if (tid == 0) {
            shared[blockIdx.x] = (int)(((long long)best << p.page_shift) / p.tile);
            const unsigned old = atom_add_release(&attn_head(p)->done, 1u);
            last = old == gridDim.x - 1;
            if (last) {
                fence_acquire();
                atomicExch(&attn_head(p)->done, 0u);
            }
        }
        __syncthreads();
        if (!last) return;
    }
    AttnItem* items = ws_ptr<AttnItem>(p.ws, p.L.item);
    const int n = p.G + p.S, per = (n + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    long long tiles = 0, units = 0, grp = 0;
    for (int i = i0; i < i1; ++i) {
        AttnItem it;
        if (i < p.G) {
            it.seq = i * p.N;
            it.tiles = __ldcg(shared + i);
            it.tile0 = 0;
            it.nodes = 0;
            int a, first = 0;
            for (int k = 0; k < p.N; ++k) {
                const int m = attn_nodes(p, it.seq + k, a);
                if (k == 0) first = a;
                if (m > 0 && a != first + it.nodes) raise_error(p.ws, kErrRange), it.nodes = 0, k = p.N;
                else it.nodes += m;
            }
            it.node0 = first;
        } else {
            it.seq = i - p.G;
            it.nodes = attn_nodes(p, it.seq, it.node0);
            const int c = attn_ctx(p, it.seq, it.nodes);
            if (c < 0) it.nodes = 0;
            it.tile0 = p.G > 0 ? __ldcg(shared + it.seq / p.N) : 0;
            it.tiles = it.nodes > 0 ? (c + it.nodes + p.tile - 1) / p.tile - it.tile0 : 0;
        }
        const int rows = it.nodes * p.gq;
        it.nrb = max(1, attn_blocks(rows, p.rb));
        it.per = max(1, min(rows, p.rb));
        if (it.nodes == 0 || it.tiles < 0) it.tiles = 0;
        const int u = it.tiles > 0 ? p.Hkv * it.nrb : 0;
        it.unit0 = u;
        it.cum = u * it.tiles;
        items[i] = it;
        tiles += it.cum;
        units += u;
        if (i < p.G) grp += u;
    }
    long long t = tiles, u = units;
    scan_pair(t, u, sa, sb);
    const long long W = sa[32];
    for (int i = i0; i < i1; ++i) {
        const long long ct = items[i].cum, cu = items[i].unit0;
        items[i].cum = (int)t;
        items[i].unit0 = (int)u;
        t += ct;
        u += cu;
    }
    __syncthreads();
    long long zero = 0;
    scan_pair(grp, zero, sa, sb);
    if (tid == 0) {
        AttnHead* h = attn_head(p);
        h->units_shared = (int)sa[32];
        const long long most = (W + p.min_tiles - 1) / p.min_tiles;
        const int n = (int)(most < p.ncta_max ? most : p.ncta_max);
        h->ncta = n;
        h->base = n > 0 ? (int)(W / n) : 0;
        h->rest = n > 0 ? (int)(W % n) : 0;
    }
}

cudaError_t launch_attn_plan(const AttnParams& p, cudaStream_t st) {
    attn_plan_kernel<<<p.G > 0 ? p.G : 1, kPlanThreads, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------------
// float32: the kernel on the FP32 pipes
// ------------------------------------------------------------------------------------------

constexpr int kSimtThreads = 128;
constexpr int kSimtKeys = 64;  // keys in a tile
constexpr int kSimtRows = 16;  // rows in a block

__device__ __forceinline__ float4 load4(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
}
template <int D>
constexpr int simt_smem() {
    return 4 * (kSimtRows * D + kSimtKeys * (D + 4) + kSimtKeys * D + kSimtKeys * (kSimtRows + 4) + 3 * kSimtRows);
}

// One block per share of the line; 16 rows x 64 keys at a time. A thread takes one key and 8 rows for
// the scores, one column (or, for D = 64, one column of half the rows) for the values. The running
// maximum m (of z / ln 2) and sum l of a row rescale what is there when the maximum grows.
template <int D>
__global__ void __launch_bounds__(kSimtThreads) attn_simt_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                                // [16][D]
    float* sk = sq + kSimtRows * D;                // [64][D + 4]
    float* sv = sk + kSimtKeys * (D + 4);          // [64][D]
    float* sp = sv + kSimtKeys * D;                // [64][16 + 4]: weights by key
    float* sm_m = sp + kSimtKeys * (kSimtRows + 4);
    float* sm_l = sm_m + kSimtRows;
    float* sm_f = sm_l + kSimtRows;
    constexpr int kP = kSimtRows + 4, kV4 = D / 4;
    constexpr int kHold = D / 8;  // rows of a thread's column: 16 (D = 128) or 8 (D = 64)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    const AttnHead* h = attn_head(p);
    const int cta = blockIdx.x;
    if (cta >= h->ncta) return;
    const AttnItem* items = ws_ptr<AttnItem>(p.ws, p.L.item);
    int x = attn_cut(h, cta);
    const int end = attn_cut(h, cta + 1);
    const int n_items = p.G + p.S;
    while (x < end) {
        const int ii = attn_find(items, n_items, x);
        const AttnItem it = items[ii];
        int next;
        const AttnPiece c = attn_piece(p, it, ii >= p.G, x, end, cta, h->units_shared, next);
        x = next;
        const int ctx = c.own ? __ldg(p.ctx_len + c.seq) : INT_MAX;
        const int keys = c.own ? ctx + it.nodes : INT_MAX;  // positions that exist
        for (int i = tid; i < kSimtRows * kV4; i += kSimtThreads) {
            const int r = i / kV4, d = (i - r * kV4) * 4;
            float4 v = make_float4(0, 0, 0, 0);
            if (r < c.rows) {
                const int row = c.row0 + r, node = row / p.gq, hq = c.hkv * p.gq + (row - node * p.gq);
                v = load4(p.q, (size_t)(c.node0 + node) * p.q_stride + (size_t)hq * D + d);
            }
            *reinterpret_cast<float4*>(sq + r * D + d) = v;
        }
        if (tid < kSimtRows) sm_m[tid] = kNegInf, sm_l[tid] = 0.0f;
        float acc[kHold];
#pragma unroll
        for (int r = 0; r < kHold; ++r) acc[r] = 0.0f;
        const int col = tid % D, vr0 = (tid / D) * kHold;
        for (int t = c.t0; t < c.t1; ++t) {
            const int pos0 = t * kSimtKeys;
            __syncthreads();
            for (int i = tid; i < kSimtKeys * kV4; i += kSimtThreads) {
                const int k = i / kV4, d = (i - k * kV4) * 4, pos = pos0 + k;
                float4 a = make_float4(0, 0, 0, 0), b = a;
                if (pos < keys) {
                    const size_t page = attn_page(p, c.seq, pos >> p.page_shift);
                    const size_t at = ((page * p.Hkv + c.hkv) * p.page_size + (pos & (p.page_size - 1))) * D + d;
                    a = load4(p.k_cache, at);
                    b = load4(p.v_cache, at);
                }
                *reinterpret_cast<float4*>(sk + k * (D + 4) + d) = a;
                *reinterpret_cast<float4*>(sv + k * D + d) = b;
            }
            __syncthreads();
            const int key = tid & (kSimtKeys - 1), r0 = (tid / kSimtKeys) * 8, pos = pos0 + key;
            float z[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) z[r] = 0.0f;
            for (int d = 0; d < D; d += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(sk + key * (D + 4) + d);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 q4 = *reinterpret_cast<const float4*>(sq + (r0 + r) * D + d);
                    z[r] = fmaf(q4.x, k4.x, z[r]);
                    z[r] = fmaf(q4.y, k4.y, z[r]);
                    z[r] = fmaf(q4.z, k4.z, z[r]);
                    z[r] = fmaf(q4.w, k4.w, z[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int row = c.row0 + r0 + r;
                bool sees = r0 + r < c.rows && pos < keys;
                if (sees && pos >= ctx) {
                    const int node = row / p.gq;
                    sees = attn_sees(p, c.node0 + node, node, pos - ctx);
                }
                sp[key * kP + r0 + r] = sees ? z[r] * p.scale2 : kNegInf;
            }
            __syncthreads();
            // statistics: a warp has 4 rows
#pragma unroll
            for (int i = 0; i < kSimtRows / 4; ++i) {
                const int r = warp * (kSimtRows / 4) + i;
                const float a = sp[lane * kP + r], b = sp[(lane + 32) * kP + r];
                const float mo = sm_m[r];
                float mx = fmaxf(a, b);
                // a NaN score makes the row NaN: fmaxf passes it over, the weight below does not
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                mx = fmaxf(mx, mo);
                const float base = mx == kNegInf ? 0.0f : mx;  // nothing seen so far: weights of zero
                const float ea = exp2f(a - base), eb = exp2f(b - base);
                float sum = ea + eb;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                sp[lane * kP + r] = ea;
                sp[(lane + 32) * kP + r] = eb;
                __syncwarp();
                if (lane == 0) {
                    const float f = mo == kNegInf ? 0.0f : exp2f(mo - base);
                    sm_f[r] = f;
                    sm_l[r] = sm_l[r] * f + sum;
                    sm_m[r] = mx;
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kHold; ++r) acc[r] *= sm_f[vr0 + r];
            // where nodes stand a weight of zero has to hide what is there, NaN too
            const bool nodes_here = pos0 + kSimtKeys > ctx;
            const int last = min(kSimtKeys, keys - pos0);
            for (int k = 0; k < last; ++k) {
                const float v = sv[k * D + col];
                const float* w = sp + k * kP + vr0;
                if (nodes_here) {
#pragma unroll
                    for (int r = 0; r < kHold; ++r)
                        if (w[r] != 0.0f) acc[r] = fmaf(w[r], v, acc[r]);
                } else {
#pragma unroll
                    for (int r = 0; r < kHold; ++r) acc[r] = fmaf(w[r], v, acc[r]);
                }
            }
        }
        __syncthreads();
        for (int r = 0; r < kHold; ++r) {
            const int rr = vr0 + r;
            if (rr >= c.rows) break;
            const int row = c.row0 + rr, node = row / p.gq, hq = c.hkv * p.gq + (row - node * p.gq);
            const size_t orow = (size_t)(c.node0 + node) * p.Hq + hq;
            const float l = sm_l[rr], m = sm_m[rr];
            if (c.whole) {
                static_cast<float*>(p.out)[orow * D + col] = l == 0.0f ? 0.0f : acc[r] / l;
                if (col == 0 && p.lse) p.lse[orow] = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718056f;
            } else {
                c.o[(size_t)rr * D + col] = acc[r];
                if (col == 0) c.ml[rr] = make_float2(m, l);
            }
        }
        __syncthreads();
    }
}

template <int D>
static cudaError_t launch_simt_t(const AttnParams& p, cudaStream_t st) {
    auto kern = attn_simt_kernel<D>;
    constexpr int smem = simt_smem<D>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ncta_max);
    cfg.blockDim = dim3(kSimtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_attn_simt(const AttnParams& p, cudaStream_t st) {
    return p.D == 64 ? launch_simt_t<64>(p, st) : launch_simt_t<128>(p, st);
}

// ------------------------------------------------------------------------------------------
// joining the pieces
// ------------------------------------------------------------------------------------------

constexpr int kJoinWarps = 8;

template <int DT>
__device__ __forceinline__ void store1(void* base, size_t i, float v) {
    if (DT == 0)
        static_cast<float*>(base)[i] = v;
    else
        static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

// Sequence that row r belongs to (ragged offsets: the last one that starts at or before it).
__device__ __forceinline__ int attn_seq_of(const AttnParams& p, int r) {
    if (!p.node_offsets) return r / p.T;
    int lo = 0, hi = p.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.node_offsets + mid) <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// One warp for each row and query head: the shared unit's pieces, then the own unit's, in the order of
// the line.
template <int DT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_combine_kernel(const __grid_constant__ AttnParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (w >= (long long)p.R * p.Hq) return;
    const int r = (int)(w / p.Hq), hq = (int)(w - (long long)r * p.Hq), hkv = hq / p.gq;
    const int s = attn_seq_of(p, r);
    const AttnHead* h = attn_head(p);
    const AttnItem* items = ws_ptr<AttnItem>(p.ws, p.L.item);
    float m = kNegInf, l = 0.0f;
    constexpr int kE = D / 32;
    float acc[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = 0.0f;
    for (int k = p.G > 0 ? 0 : 1; k < 2; ++k) {
        const AttnItem it = items[k == 0 ? s / p.N : p.G + s];
        if (it.tiles == 0) continue;
        const int node = r - it.node0;
        if (node < 0 || node >= it.nodes) return;  // bad offsets, already reported
        const int row = node * p.gq + (hq - hkv * p.gq), rb = row / it.per, rr = row - rb * it.per;
        const int u = hkv * it.nrb + rb;
        const int x0 = it.cum + u * it.tiles;
        const int c0 = attn_cta_of(h, x0), c1 = attn_cta_of(h, x0 + it.tiles - 1);
        if (k == 1 && it.tile0 == 0 && c0 == c1) return;  // written directly
        for (int c = c0; c <= c1; ++c) {
            const size_t slot = k == 0 ? (size_t)(it.unit0 + u + c) : (size_t)(it.unit0 + u - h->units_shared + c);
            const size_t at = slot * (k == 0 ? p.L.rows_g : p.L.rows_s) + rr;
            const float2 ml = __ldcg(ws_ptr<float2>(p.ws, k == 0 ? p.L.ml_g : p.L.ml_s) + at);
            const float* o = ws_ptr<float>(p.ws, k == 0 ? p.L.slot_g : p.L.slot_s) + at * D;
            float v[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] = __ldcg(o + e * 32 + lane);
            if (ml.y == 0.0f) continue;  // saw nothing
            const float mx = fmaxf(m, ml.x);
            const float base = mx == kNegInf ? 0.0f : mx;
            const float fa = l == 0.0f ? 0.0f : exp2f(m - base), fb = exp2f(ml.x - base);
            l = l * fa + ml.y * fb;
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[e] = fmaf(acc[e], fa, v[e] * fb);
            m = mx;
        }
    }
    const size_t orow = (size_t)r * p.Hq + hq;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < kE; ++e) store1<DT>(p.out, orow * D + e * 32 + lane, acc[e] * inv);
    if (lane == 0 && p.lse) p.lse[orow] = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718056f;
}

template <int DT, int D>
static cudaError_t launch_combine_t(const AttnParams& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((long long)p.R * p.Hq + kJoinWarps - 1) / kJoinWarps));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_combine_kernel<DT, D>, p);
}

cudaError_t launch_attn_combine(const AttnParams& p, int dtype, cudaStream_t st) {
    if (p.D == 64) return dtype == 0 ? launch_combine_t<0, 64>(p, st) : launch_combine_t<1, 64>(p, st);
    return dtype == 0 ? launch_combine_t<0, 128>(p, st) : launch_combine_t<1, 128>(p, st);
}

}  // namespace smcsd
