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

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ long long plan_prefix(long long v, long long* sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += t;
    }
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    long long w = lane < kPlanThreads / 32 ? sums[lane] : 0, before = w;
#pragma unroll
    for (int o = 1; o < kPlanThreads / 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
    }
    total = __shfl_sync(0xffffffffu, before, kPlanThreads / 32 - 1);
    return __shfl_sync(0xffffffffu, before - w, warp) + in - v;
}

// Item i without its places on the line.
__device__ __forceinline__ AttnItem plan_item(const AttnParams& p, const int* shared, int i) {
    AttnItem it;
    if (i < p.G) {
        it.seq = i * p.N;
        it.keys = __ldcg(shared + i);
        it.tiles = (it.keys + (1 << p.log_tile) - 1) >> p.log_tile;
        it.key0 = 0;
        int first, a;
        it.nodes = attn_nodes(p, it.seq, first);
        for (int k = 1; k < p.N; ++k) {
            const int m = attn_nodes(p, it.seq + k, a);
            if (m > 0 && a != first + it.nodes) {  // offsets that do not fit, already reported
                it.nodes = 0;
                break;
            }
            it.nodes += m;
        }
        it.node0 = first;
    } else {
        it.seq = i - p.G;
        it.nodes = attn_nodes(p, it.seq, it.node0);
        const int c = attn_ctx(p, it.seq, it.nodes);
        if (c < 0) it.nodes = 0;
        it.key0 = p.G > 0 ? __ldcg(shared + it.seq / p.N) : 0;
        it.tiles = it.nodes > 0 ? (c + it.nodes - it.key0 + (1 << p.log_tile) - 1) >> p.log_tile : 0;
        it.keys = 0;
    }
    it.pad[0] = it.pad[1] = 0;
    return it;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnParams p) {
    __shared__ int best;
    __shared__ unsigned last;
    __shared__ long long sums[kPlanThreads / 32];
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    int* shared = ws_ptr<int>(p.ws, p.L.shared);
    if (p.G > 0) {
        // pages that every sequence of the group has at the same place, all of them full context; four threads have a
        // column, a quarter of the sequences each
        const int s0 = blockIdx.x * p.N;
        if (tid == 0) best = p.pages_per_seq;
        __syncthreads();
        for (int i = tid; i < p.N; i += kPlanThreads) atomicMin(&best, max(0, __ldg(p.ctx_len + s0 + i)) >> p.page_shift);
        __syncthreads();
        const int lim = best;
        __syncthreads();
        const int32_t* row = p.table + (long long)s0 * p.pages_per_seq;
        for (int j = tid & 127; j < lim && j < *reinterpret_cast<volatile int*>(&best); j += 128) {
            const int id = __ldg(row + j);
            bool same = id >= 0;
#pragma unroll 4
            for (int k = 1 + (tid >> 7); k < p.N; k += kPlanThreads / 128) same &= __ldg(row + (long long)k * p.pages_per_seq + j) == id;
            if (!same) atomicMin(&best, j);
        }
        __syncthreads();
        if (tid == 0) {
            // less than a tile is not worth a unit of its own
            const int keys = best << p.page_shift;
            shared[blockIdx.x] = keys >> p.log_tile ? keys : 0;
            unsigned* done = ws_ptr<unsigned>(p.ws, kFrontPlanned);
            last = atom_add_release(done, 1u) == gridDim.x - 1;
            if (last) {
                fence_acquire();
                atomicExch(done, 0u);
            }
        }
        __syncthreads();
        if (!last) return;
    }
    // places (high word) and units (low word) before each item: a thread has a run of them
    AttnItem* items = ws_ptr<AttnItem>(p.ws, p.L.item);
    const int n = p.G + p.S, per = (n + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    AttnItem it;
    // by cost; where that leaves blocks less than a tile's places, with a place for each tile
    AttnCost cost(p, true);
    long long at, total;
    bool weighted = true;
    for (;;) {
        long long mine = 0;
        for (int i = i0; i < i1; ++i) {
            it = plan_item(p, shared, i);
            const long long u = attn_units(p, it);
            mine += ((long long)cost.item(p, it) << 32) + u;
        }
        at = plan_prefix(mine, sums, total);
        if (!weighted || AttnCost::fits(p, total >> 32)) break;
        weighted = false;
        cost = AttnCost(p, false);
        __syncthreads();  // the sums have been read
    }
    for (int i = i0; i < i1; ++i) {
        if (per > 1) it = plan_item(p, shared, i);
        const long long u = attn_units(p, it);
        it.cum = (int)(at >> 32);
        it.unit0 = (int)(at & 0xffffffffll);
        items[i] = it;
        at += ((long long)cost.item(p, it) << 32) + u;
        if (i == p.G - 1) attn_head(p)->units_shared = (int)(at & 0xffffffffll);
    }
    if (tid == 0) {
        AttnHead* h = attn_head(p);
        const int W = (int)(total >> 32);
        const AttnCut cut(p, W);
        if (p.G == 0) h->units_shared = 0;
        h->weighted = weighted;
        h->ncta = cut.ncta;
        h->base = cut.base;
        h->rest = cut.rest;
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

// Two blocks per SM, one share of the line each; 16 rows x 64 keys at a time. Latency bounds it at the sizes that float32 is
// for (six barriers a tile): 16 us for 4 trees of three nodes over 1000 tokens, 8 heads on 4 of 64 columns.
// A thread takes one key and 8 rows for
// the scores, one column (or, for D = 64, one column of half the rows) for the values. The running
// maximum m (of z / ln 2) and sum l of a row rescale what is there when the maximum grows.
template <int D, bool kPlanned>
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
    __shared__ PieceInfo s_piece, s_pending[2];
    __shared__ int s_last[2];
    int pending = 0;
    Walker<kPlanned> walk;
    if (warp == 0) walk.begin(p, lane);
    for (;;) {
        if (warp == 0) {
            PieceInfo c;
            walk.next(p, c, lane);
            if (lane == 0) s_piece = c;
        }
        __syncthreads();
        const PieceInfo c = s_piece;
        if (c.rows == 0) break;
        const int ctx = c.ctx, keys = c.end;  // positions that exist
        for (int i = tid; i < kSimtRows * kV4; i += kSimtThreads) {
            const int r = i / kV4, d = (i - r * kV4) * 4;
            float4 v = make_float4(0, 0, 0, 0);
            if (r < c.rows) {
                const int row = c.row0 + r, node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
                v = load4(p.q, (size_t)(c.node0 + node) * p.q_stride + (size_t)hq * D + d);
            }
            *reinterpret_cast<float4*>(sq + r * D + d) = v;
        }
        if (tid < kSimtRows) sm_m[tid] = kNegInf, sm_l[tid] = 0.0f;
        float acc[kHold];
#pragma unroll
        for (int r = 0; r < kHold; ++r) acc[r] = 0.0f;
        const int col = tid % D, vr0 = (tid / D) * kHold;
        for (int t = 0; t < c.n; ++t) {
            const int pos0 = c.key0 + t * kSimtKeys;
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
                    const int node = attn_node(p, row);
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
            const int row = c.row0 + rr, node = attn_node(p, row), hq = c.hkv * p.gq + (row - node * p.gq);
            const size_t orow = (size_t)(c.node0 + node) * p.Hq + hq;
            const float l = sm_l[rr], m = sm_m[rr];
            if (c.whole) {
                static_cast<float*>(p.out)[orow * D + col] = l == 0.0f ? 0.0f : acc[r] / l;
                if (col == 0 && p.lse) p.lse[orow] = attn_lse(m, l);
            } else {
                c.o[(size_t)rr * D + col] = acc[r];
                if (col == 0) c.ml[rr] = make_float2(m, l);
            }
        }
        if (c.join > 0) {
            if (tid == 0) s_pending[pending] = c;
            ++pending;
        }
        __syncthreads();
    }
    if (!kPlanned && pending > 0) attn_join_last<0, D, 1, 4>(p, s_pending, pending, tid, kSimtThreads, s_last, [] { __syncthreads(); });
}

template <int D>
static cudaError_t launch_simt_t(const AttnParams& p, cudaStream_t st) {
    auto kern = p.planned ? attn_simt_kernel<D, true> : attn_simt_kernel<D, false>;
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
    cfg.numAttrs = p.planned ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_attn_simt(const AttnParams& p, cudaStream_t st) {
    return p.D == 64 ? launch_simt_t<64>(p, st) : launch_simt_t<128>(p, st);
}

// ------------------------------------------------------------------------------------------
// joining the pieces after the planning kernel
// ------------------------------------------------------------------------------------------

constexpr int kJoinThreads = 256;

// The slots of one row's pieces of a unit, from the i-th on: one after the other with groups, otherwise every second one from
// the second piece on.
struct JoinRun {
    const float* o;
    const float2* ml;
    size_t rows;  // of a slot
    int count;
    template <bool kGroups>
    __device__ __forceinline__ size_t at(int i) const {
        return (kGroups || i == 0 ? i : 2 * i - 1) * rows;
    }
};

// After the planning kernel: a few blocks (z) for each sequence (x) and unit of it (y). A row's pieces are joined in the
// order of the line, the shared unit's first: a warp has a row (of 64 columns: two), four columns a thread, and the first two
// pieces of both units are loaded together.
template <int DT, int D, bool kGroups>
__global__ void __launch_bounds__(kJoinThreads) attn_combine_kernel(const __grid_constant__ AttnParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AttnHead* h = attn_head(p);
    const AttnItem* items = ws_ptr<AttnItem>(p.ws, p.L.item);
    AttnCut cut;
    cut.base = h->base;
    cut.rest = h->rest;
    const AttnCost cost(p, h->weighted);
    const AttnItem it = items[p.G + blockIdx.x], grp = items[kGroups ? blockIdx.x / p.N : 0];
    if (it.tiles == 0) return;
    const bool shared = kGroups && grp.tiles > 0;
    constexpr int kLanes = D / 4, kRows = 32 / kLanes;  // lanes of a row, rows of a warp at a time
    const int col = (lane % kLanes) * 4;
    const int step = gridDim.z * (kJoinThreads / 32) * kRows;
    // Where the unit's pieces are is worked out once a block: its own, and those of the one or two row blocks of the shared
    // unit that its rows lie in (with each thread's own divisions the kernel's instructions bound it).
    __shared__ JoinRun s_run[3];
#pragma unroll 1
    for (int u = blockIdx.y; u < p.Hkv * it.nrb; u += gridDim.y) {
        const int hkv = it.nrb == 1 ? u : u / it.nrb, row0 = (u - hkv * it.nrb) * it.per, rows = min(it.per, it.nodes * p.gq - row0);
        const int gr0 = row0 + (it.node0 - grp.node0) * p.gq, grb0 = shared ? gr0 / grp.per : 0;
        if (threadIdx.x < 3) {
            const bool own = threadIdx.x == 0;
            const AttnItem& of = own ? it : grp;
            const int rb = own ? u - hkv * it.nrb : grb0 + (int)threadIdx.x - 1;
            JoinRun r{nullptr, nullptr, 0, 0};
            if (own || (shared && rb < grp.nrb)) {
                const int its = min(of.per, of.nodes * p.gq - rb * of.per);
                const int x0 = of.cum + hkv * cost.head(p, of) + rb * cost.unit(of.per, of.tiles) + cost.empty;  // its first tile's place
                const int c0 = cut.block(x0);
                r.rows = own ? p.L.rows_s : p.L.rows_g;
                const size_t at = (size_t)(kGroups ? of.unit0 + hkv * of.nrb + rb - (own ? h->units_shared : 0) + c0 : 2 * c0 + 1) * r.rows;
                r.o = ws_ptr<float>(p.ws, own ? p.L.slot_s : p.L.slot_g) + at * D;
                r.ml = ws_ptr<float2>(p.ws, own ? p.L.ml_s : p.L.ml_g) + at;
                r.count = cut.block(x0 + (of.tiles - 1) * cost.tile(its)) - c0 + 1;
            }
            s_run[threadIdx.x] = r;
        }
        __syncthreads();
        const bool direct = !shared && s_run[0].count == 1;  // written by the pass itself
#pragma unroll 1
        for (int r = (blockIdx.z * (kJoinThreads / 32) + warp) * kRows + lane / kLanes; r < rows && !direct; r += step) {
            const int row = row0 + r, n = attn_node(p, row);
            JoinRun run[2];
            run[0].count = 0;
            if (shared) {
                int at = gr0 + r - grb0 * grp.per;
                const bool next = at >= grp.per;
                at -= next ? grp.per : 0;
                run[0] = s_run[1 + next];
                run[0].o += (size_t)at * D;
                run[0].ml += at;
            }
            run[1] = s_run[0];
            run[1].o += (size_t)r * D;
            run[1].ml += r;
            float2 s[4];
            float4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const JoinRun& of = run[x >> 1];
                s[x] = make_float2(0, 0);
                v[x] = make_float4(0, 0, 0, 0);
                if ((x & 1) < of.count) {
                    s[x] = __ldcg(of.ml + of.at<kGroups>(x & 1));
                    v[x] = __ldcg(reinterpret_cast<const float4*>(of.o + of.at<kGroups>(x & 1) * D + col));
                }
            }
            AttnJoin j;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                j.add(s[x], v[x]);
                if (x & 1) {
#pragma unroll 2
                    for (int i = 2; i < run[x >> 1].count; ++i)
                        j.add(__ldcg(run[x >> 1].ml + run[x >> 1].at<kGroups>(i)),
                              __ldcg(reinterpret_cast<const float4*>(run[x >> 1].o + run[x >> 1].at<kGroups>(i) * D + col)));
                }
            }
            j.store<DT, D>(p, (size_t)(it.node0 + n) * p.Hq + hkv * p.gq + (row - n * p.gq), col);
        }
        __syncthreads();  // the unit's pieces have been read
    }
}

template <int DT, int D>
static cudaError_t launch_combine_t(const AttnParams& p, cudaStream_t st) {
    // a warp takes one row (four rows each, loads of its pieces one after the other: 21 us in place of 17, with cold caches, for
    // 1024 units of 20 rows)
    const long long rows = (long long)p.T * p.gq, units = (long long)p.Hkv * attn_blocks(rows, 1 << p.log_rb);
    const unsigned parts = (unsigned)((rows < (1 << p.log_rb) ? rows : (1 << p.log_rb)) + 7) / 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.S, (unsigned)(units < 65535 ? units : 65535), parts);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.G > 0 ? attn_combine_kernel<DT, D, true> : attn_combine_kernel<DT, D, false>, p);
}

cudaError_t launch_attn_combine(const AttnParams& p, int dtype, cudaStream_t st) {
    if (p.D == 64) return dtype == 0 ? launch_combine_t<0, 64>(p, st) : launch_combine_t<1, 64>(p, st);
    return dtype == 0 ? launch_combine_t<0, 128>(p, st) : launch_combine_t<1, 128>(p, st);
}

}  // namespace smcsd
