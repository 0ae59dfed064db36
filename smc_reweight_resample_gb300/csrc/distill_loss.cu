// distill_loss.cu -- a draft's loss against a teacher's top logits, and its gradient, in one pass over the logits.
//
// q = softmax(c z) over the vocabulary, c = 1 / temperature; p the teacher's probabilities of the row's listed tokens, p_r what they
// leave to the rest (0 where the list is taken for everything):
//   loss = sum_k p_k (log p_k - log q_k) + p_r (log p_r - log q_r),     q_r = sum of q over the tokens that are not listed;
//   dloss / dz_v = c (P q_v - p_v) for a listed v,  c q_v (P - p_r / q_r) for others,     P = sum p + p_r.
// A row is read once: a cluster of blocks holds it in shared memory, its listed tokens are taken out of it (their sum is kept apart,
// so that q_r is a sum and no difference), the blocks' maxima and sums meet in the cluster's shared memories, and each block writes
// its share of the gradient from what it holds.
#include <cooperative_groups.h>

#include "ops_launch.cuh"
#include "smcsd_launch.cuh"

namespace cg = cooperative_groups;

namespace smcsd {

constexpr int kDistillThreads = 256;
constexpr int kDistillWarps = kDistillThreads / 32;
static_assert(kDistillThreads >= kDistillMostTokens, "a thread for each listed token");

__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int DT>
struct Elem;
template <>
struct Elem<0> {
    using T = uint32_t;
};
template <>
struct Elem<1> {
    using T = unsigned short;
};
template <int DT>
__device__ __forceinline__ uint32_t round_to(float f) {
    if (DT == 0) return __float_as_uint(f);
    unsigned short r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
}
template <int DT>
__device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == 0)
            w[i] = __float_as_uint(f[i]);
        else
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ void unpack_vec(const uint4& x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == 0) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

struct DistillShared {
    int token[kDistillMostTokens];
    float p[kDistillMostTokens];
    float z[kDistillMostTokens];       // in the first block: the listed tokens' logits
    float4 part[kDistillMostCtas];     // of each block: maximum and sum of the rest, of the listed tokens
    float a[kDistillWarps], b[kDistillWarps];
    dd d[kDistillWarps];
};

// Maxima, or sums, of two values over the block.
__device__ __forceinline__ float2 block_max2(DistillShared& s, float a, float b) {
    a = warp_max(a);
    b = warp_max(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.a[threadIdx.x >> 5] = a, s.b[threadIdx.x >> 5] = b;
    __syncthreads();
    a = s.a[0], b = s.b[0];
#pragma unroll
    for (int w = 1; w < kDistillWarps; ++w) a = fmaxf(a, s.a[w]), b = fmaxf(b, s.b[w]);
    return make_float2(a, b);
}
__device__ __forceinline__ float2 block_sum2(DistillShared& s, float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.a[threadIdx.x >> 5] = a, s.b[threadIdx.x >> 5] = b;
    __syncthreads();
    a = s.a[0], b = s.b[0];
#pragma unroll
    for (int w = 1; w < kDistillWarps; ++w) a += s.a[w], b += s.b[w];
    return make_float2(a, b);
}
__device__ __forceinline__ dd block_sum_dd(DistillShared& s, dd a) {
    a = warp_sum_dd(a);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.d[threadIdx.x >> 5] = a;
    __syncthreads();
    a = s.d[0];
#pragma unroll
    for (int w = 1; w < kDistillWarps; ++w) a = dd_add(a, s.d[w]);
    return a;
}

// This block's share of a row: vectors first .. first + n - 1 of the row's aligned vectors, the first of which begins `shift`
// elements before the row.
template <int DT>
struct Share {
    const char* row;
    int shift, V;
    long long first;
    int n;
    // the elements of vector i of the share that lie in the row: from lo to hi - 1
    __device__ void within(int i, int& lo, int& hi) const {
        constexpr int PV = Geo<DT>::kPerVec;
        const long long e = (first + i) * PV - shift;
        lo = e < 0 ? (int)-e : 0;
        hi = e + PV > V ? (int)(V - e) : PV;
    }
    __device__ long long element(int i) const { return (first + i) * (long long)Geo<DT>::kPerVec - shift; }
};

// Writes f(i) (a vector of elements) for every vector i of the share to the row of the gradient.
template <int DT, typename F>
__device__ __forceinline__ void write_share(const Share<DT>& h, char* out, F&& f) {
    constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes;
    using T = typename Elem<DT>::T;
    const bool alike = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(h.row)) & 15u) == 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < h.n; i += kDistillThreads) {
        int lo, hi;
        h.within(i, lo, hi);
        const uint4 x = f(i);
        char* to = out + h.element(i) * B;
        if (alike && lo == 0 && hi == PV) {
            *reinterpret_cast<uint4*>(to) = x;
        } else {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < PV; ++e)
                if (e >= lo && e < hi) reinterpret_cast<T*>(to)[e] = (T)(DT == 0 ? w[e & 3] : w[(e >> 1) & 3] >> (16 * (e & 1)));
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kDistillThreads) distill_kernel(const __grid_constant__ DistillParams p) {
    constexpr int PV = Geo<DT>::kPerVec, B = Geo<DT>::kBytes;
    using T = typename Elem<DT>::T;
    extern __shared__ uint4 s_row[];
    __shared__ DistillShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = p.ctas, rank = (int)cl.block_rank(), tid = threadIdx.x;
    const int r = blockIdx.x / C;
    auto started = cl.barrier_arrive();  // the other blocks' shared memory may be written once all have come here

    // the row's list
    int token = -1;
    float value = kNegInf;
    if (tid < p.K) {
        token = __ldg(p.tokens + (long long)r * p.K + tid);
        value = __ldg(p.values + (long long)r * p.K + tid);
        if (token < 0 || token >= p.V) {
            if (token != -1) raise_error(p.ws, kErrRange);
            token = -1;
            value = kNegInf;
        } else if (!(value < kPosInf)) {
            raise_error(p.ws, kErrNonfinite);
        }
    }
    if (tid < kDistillMostTokens) s.token[tid] = token;
    const float weight = p.weight ? __ldg(p.weight + r) : 1.0f;

    Share<DT> h;
    h.row = static_cast<const char*>(p.logits) + (long long)r * p.row_stride * B;
    h.shift = (int)(reinterpret_cast<uintptr_t>(h.row) & 15u) / B;
    h.V = p.V;
    h.first = (long long)rank * p.vecs;
    const long long all = ((long long)p.V + h.shift + PV - 1) / PV;
    h.n = (int)(all - h.first < 0 ? 0 : all - h.first < p.vecs ? all - h.first : p.vecs);
    char* out = p.grad ? static_cast<char*>(p.grad) + (long long)r * p.grad_stride * B : nullptr;

    const bool some = __syncthreads_or(value > kNegInf);
    if (!some || (weight == 0.0f && !p.loss)) {
        cl.barrier_wait(std::move(started));
        if (out) write_share<DT>(h, out, [](int) { return make_uint4(0, 0, 0, 0); });
        if (rank == 0 && tid == 0 && p.loss) p.loss[r] = 0.0f;
        return;
    }

    // the share's whole vectors on their way; the row's first and last vector may lie in it in part
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(s_row);
    for (int i = tid; i < h.n; i += kDistillThreads) {
        int lo, hi;
        h.within(i, lo, hi);
        if (lo == 0 && hi == PV) {
            copy16_async(to + 16u * i, h.row + h.element(i) * B);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = DT == 0 ? neg_inf_bits<0>() : neg_inf_bits<1>() * 0x10001u;
#pragma unroll
            for (int e = 0; e < PV; ++e)
                if (e >= lo && e < hi) {
                    const uint32_t bits = logit_bits<DT>(h.row, h.element(i) + e);
                    if (DT == 0)
                        w[e & 3] = bits;
                    else
                        w[(e >> 1) & 3] = e & 1 ? (w[(e >> 1) & 3] & 0xffffu) | bits << 16 : (w[(e >> 1) & 3] & 0xffff0000u) | bits;
                }
            s_row[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }

    // meanwhile the teacher's probabilities
    float logp, prob, rest = 0.0f, mass = 1.0f;
    if (p.rest) {
        logp = value;
        prob = value > kNegInf ? expf(value) : 0.0f;
        const dd sum = block_sum_dd(s, dd{prob, 0.0f});
        rest = fmaxf(dd_add(dd{1.0f, 0.0f}, dd_neg(sum)).hi, 0.0f);
        mass = fmaxf(sum.hi, 1.0f);
    } else {
        const float top = block_max2(s, value, kNegInf).x;
        const float e = value > kNegInf ? expf(value - top) : 0.0f;
        const dd sum = block_sum_dd(s, dd{e, 0.0f});
        logp = value - top - logf(sum.hi);
        prob = e / sum.hi;
    }
    if (tid < kDistillMostTokens) s.p[tid] = prob;
    __syncthreads();
    // a token that is listed several times: its first place stands for all of them
    bool first = token >= 0;
    float listed = 0.0f;
    if (token >= 0)
        for (int k = 0; k < p.K; ++k)
            if (s.token[k] == token) {
                listed += s.p[k];
                first = first && k >= tid;
            }

    copies_done();
    __syncthreads();
    // the listed tokens are taken out of the share
    T* elems = reinterpret_cast<T*>(s_row);
    const long long at = token + (long long)h.shift - h.first * PV;
    const bool mine = token >= 0 && at >= 0 && at < (long long)h.n * PV;
    float z = kNegInf;
    if (mine) z = bits_to_float<DT>((uint32_t)elems[at]);
    __syncthreads();
    if (mine) elems[at] = (T)neg_inf_bits<DT>();
    __syncthreads();

    // the share's maximum and sum
    float m = kNegInf;
    for (int i = tid; i < h.n; i += kDistillThreads) {
        float f[PV];
        unpack_vec<DT>(s_row[i], f);
#pragma unroll
        for (int e = 0; e < PV; ++e) m = fmaxf(m, f[e]);
    }
    const float2 top = block_max2(s, m, first ? z : kNegInf);
    float sum = 0.0f;
    const float m0 = top.x > kNegInf ? top.x : 0.0f;  // a share of -inf alone adds up to 0, one with NaN to NaN
    for (int i = tid; i < h.n; i += kDistillThreads) {
        float f[PV];
        unpack_vec<DT>(s_row[i], f);
#pragma unroll
        for (int e = 0; e < PV; ++e) f[e] = exp2_fast((f[e] - m0) * p.c2);
#pragma unroll
        for (int o = PV / 2; o > 0; o >>= 1)
#pragma unroll
            for (int e = 0; e < o; ++e) f[e] += f[e + o];
        sum += f[0];
    }
    const float ez = first && mine ? (top.y > kNegInf ? exp2f((z - top.y) * p.c2) : z != z ? z : 0.0f) : 0.0f;
    const float2 total = block_sum2(s, sum, ez);

    cl.barrier_wait(std::move(started));
    if (mine) *cl.map_shared_rank(&s.z[tid], 0) = z;
    if (tid < C) *cl.map_shared_rank(&s.part[rank], tid) = make_float4(top.x, total.x, top.y, total.y);
    cl.sync();

    // the row's
    float mr = kNegInf, mt = kNegInf;
    for (int k = 0; k < C; ++k) mr = fmaxf(mr, s.part[k].x), mt = fmaxf(mt, s.part[k].z);
    float sr = 0.0f, st = 0.0f;
    for (int k = 0; k < C; ++k) {
        const float4 x = s.part[k];
        sr += x.x > kNegInf ? x.y * exp2f((x.x - mr) * p.c2) : x.y;
        st += x.z > kNegInf ? x.w * exp2f((x.z - mt) * p.c2) : x.w;
    }
    const float mm = fmaxf(mr, mt);
    const float kr = mr > kNegInf ? exp2f((mr - mm) * p.c2) : 0.0f, kt = mt > kNegInf ? exp2f((mt - mm) * p.c2) : 0.0f;
    const float S = sr * kr + st * kt;
    if (rank == 0) {
        if (tid == 0 && !(S > 0.0f && S < kPosInf)) raise_error(p.ws, kErrNonfinite);
        if (p.loss) {
            const float ls = logf(S);
            float term = 0.0f;
            if (prob > 0.0f) term = prob * (logp - ((s.z[tid] - mm) * p.c - ls));
            if (tid == 0 && rest > 0.0f) term += rest * (logf(rest) - (logf(sr) + (mr - mm) * p.c - ls));
            const float loss = block_sum2(s, term, 0.0f).x;
            if (tid == 0) p.loss[r] = loss;
        }
    }
    if (!out) return;
    const float wc = weight * p.c;
    // a rest without mass (all -inf) gets no gradient
    const float scale = mr > kNegInf ? wc * (mass * (kr / S) - rest / sr) : 0.0f;
    const float m1 = mr > kNegInf ? mr : 0.0f;
    write_share<DT>(h, out, [&](int i) {
        float f[PV];
        unpack_vec<DT>(s_row[i], f);
#pragma unroll
        for (int e = 0; e < PV; ++e) f[e] = exp2_fast((f[e] - m1) * p.c2) * scale;
        return pack<DT>(f);
    });
    __syncthreads();  // the listed tokens' places have been written as part of the rest
    if (mine && first) {
        const float q = exp2f((z - mm) * p.c2) / S;
        reinterpret_cast<T*>(out)[token] = (T)round_to<DT>(wc * (mass * q - listed));
    }
}

cudaError_t launch_distill(const DistillParams& p0, int dtype, cudaStream_t st) {
    DistillParams p = p0;
    // shares of at most 32 KB, so that several rows' blocks are in an SM at a time
    const long long bytes = (long long)p.V * (dtype == 0 ? 4 : 2), vecs = (bytes + 30) / 16;
    p.ctas = 1;
    while (p.ctas < kDistillMostCtas && vecs > p.ctas * 2048ll) p.ctas *= 2;
    p.vecs = (int)((vecs + p.ctas - 1) / p.ctas);
    const size_t shared = 16 * (size_t)p.vecs;
    const auto kernel = dtype == 0 ? distill_kernel<0> : distill_kernel<1>;
    cudaError_t e = cudaSuccess;
    if (shared > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.R * p.ctas));
    cfg.blockDim = dim3(kDistillThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace smcsd
