// logits_process.cu -- penalties for repeated tokens, biases and grammar masks on logits.
//
// One block per sequence and slice of the vocabulary: it counts the slice's tokens of the sequence's
// history in shared memory once, notes the biases, and streams the slice of all of the sequence's
// rows past them.
#include <cuda_bf16.h>

#include "serve_launch.cuh"
#include "smcsd_launch.cuh"

namespace smcsd {

constexpr int kLogThreads = 256;
constexpr int kLogWarps = kLogThreads / 32;
constexpr int kSlice = 4096;    // tokens of a block
constexpr int kSegment = 1024;  // tokens of a warp at a time

template <int DT>
__device__ __forceinline__ uint32_t to_bits(float z) {
    if (DT == 0) return __float_as_uint(z);
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(z));
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kLogThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
    __shared__ int s_count[kSlice];
    __shared__ int s_bias[kSlice];               // 1 + index of the last bias entry of a token
    __shared__ uint32_t s_hit[kSlice / 32];      // tokens with a count or a bias
    __shared__ uint32_t s_path[kLogWarps][kSegment / 32];  // tokens of a row's own path
    constexpr int kE = Geo<DT>::kPerVec;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.y, lo = blockIdx.x * kSlice, len = min(kSlice, p.V - lo);
    int first;
    const int n = nodes_of(p.n, s, first, p.ws);
    for (int i = tid; i < kSlice; i += kLogThreads) s_count[i] = 0, s_bias[i] = 0;
    for (int i = tid; i < kSlice / 32; i += kLogThreads) s_hit[i] = 0;
    __syncthreads();
    if (p.hist_tokens) {
        const int a = __ldg(p.hist_offsets + s), b = __ldg(p.hist_offsets + s + 1);
        if (a < 0 || b < a || b > p.n_hist) {
            raise_error(p.ws, kErrRange);
        } else {
            for (int i = a + tid; i < b; i += kLogThreads) {
                const int tok = __ldg(p.hist_tokens + i), k = tok - lo;
                if (k >= 0 && k < len) {
                    atomicAdd(&s_count[k], 1);
                    atomicOr(&s_hit[k >> 5], 1u << (k & 31));
                } else if (tok < -1 || tok >= p.V) {
                    raise_error(p.ws, kErrRange);
                }
            }
        }
    }
    int b0 = 0;
    if (p.bias_tokens) {
        b0 = __ldg(p.bias_offsets + s);
        const int b = __ldg(p.bias_offsets + s + 1);
        if (b0 < 0 || b < b0 || b > p.n_bias) {
            raise_error(p.ws, kErrRange);
        } else {
            for (int i = b0 + tid; i < b; i += kLogThreads) {
                const int tok = __ldg(p.bias_tokens + i), k = tok - lo;
                if (k >= 0 && k < len) {
                    atomicMax(&s_bias[k], i - b0 + 1);
                    atomicOr(&s_hit[k >> 5], 1u << (k & 31));
                } else if (tok < -1 || tok >= p.V) {
                    raise_error(p.ws, kErrRange);
                }
            }
        }
    }
    __syncthreads();
    const float rep = p.repetition ? __ldg(p.repetition + s) : 1.0f;
    const float pres = p.presence ? __ldg(p.presence + s) : 0.0f;
    const float freq = p.frequency ? __ldg(p.frequency + s) : 0.0f;
    const bool in_place = p.out == p.logits;
    const int segs = (len + kSegment - 1) / kSegment;
    for (int unit = warp; unit < n * segs; unit += kLogWarps) {
        const int t = unit / segs, g0 = (unit - t * segs) * kSegment, glen = min(kSegment, len - g0);
        const long long row = first + t;
        // the tokens that the row's path holds in this segment
        uint32_t* path = s_path[warp];
        path[lane] = 0;
        __syncwarp();
        if (p.node_tokens) {
            const int upto = p.mask ? n : t + 1;
            for (int j = lane; j < upto; j += 32) {
                if (p.mask && !((__ldg(p.mask + row * p.words + (j >> 5)) >> (j & 31)) & 1u)) continue;
                const int tok = __ldg(p.node_tokens + first + j), k = tok - lo - g0;
                if (k >= 0 && k < glen)
                    atomicOr(&path[k >> 5], 1u << (k & 31));
                else if (tok < -1 || tok >= p.V)
                    raise_error(p.ws, kErrRange);
            }
        }
        __syncwarp();
        const char* src = static_cast<const char*>(p.logits) + (row * p.V + lo + g0) * Geo<DT>::kBytes;
        char* dst = static_cast<char*>(p.out) + (row * p.V + lo + g0) * Geo<DT>::kBytes;
        const uint32_t* allow = p.allowed ? p.allowed + row * p.allowed_words + ((lo + g0) >> 5) : nullptr;
        for (int e0 = lane * kE; e0 < glen; e0 += 32 * kE) {
            uint32_t raw[4] = {0, 0, 0, 0};
            const int cnt = min(kE, glen - e0);
            if (VEC) {
                const uint4 v = *reinterpret_cast<const uint4*>(src + (size_t)e0 * Geo<DT>::kBytes);
                raw[0] = v.x, raw[1] = v.y, raw[2] = v.z, raw[3] = v.w;
            } else {
                for (int e = 0; e < cnt; ++e) {
                    const uint32_t b = logit_bits<DT>(src, e0 + e);
                    if (DT == 0)
                        raw[e] = b;
                    else
                        raw[e >> 1] |= b << ((e & 1) * 16);
                }
            }
            const int sh = e0 & 31;
            const uint32_t full = (1u << kE) - 1u;
            const uint32_t on_path = (path[e0 >> 5] >> sh) & full;
            uint32_t hit = (s_hit[(g0 + e0) >> 5] >> sh) & full;
            hit |= on_path;
            uint32_t ok = allow ? (__ldg(allow + (e0 >> 5)) >> sh) & full : full;
            hit &= ok;
            if (hit) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    if (!((hit >> e) & 1u)) continue;
                    const int k = g0 + e0 + e, tok = lo + k;
                    int count = s_count[k];
                    if ((on_path >> e) & 1u) {
                        const int upto = p.mask ? n : t + 1;
                        for (int j = 0; j < upto; ++j) {
                            if (p.mask && !((__ldg(p.mask + row * p.words + (j >> 5)) >> (j & 31)) & 1u)) continue;
                            count += __ldg(p.node_tokens + first + j) == tok;
                        }
                    }
                    const uint32_t w = DT == 0 ? raw[e & 3] : (raw[e >> 1] >> ((e & 1) * 16)) & 0xffffu;
                    float z = bits_to_float<DT>(w);
                    if (count > 0) {
                        z = z > 0.0f ? z / rep : z * rep;
                        z = z - freq * (float)count;
                        z = z - pres;
                    }
                    const int bi = s_bias[k];
                    if (bi) z = z + __ldg(p.bias_values + b0 + bi - 1);
                    const uint32_t b = to_bits<DT>(z);
                    if (DT == 0)
                        raw[e & 3] = b;
                    else
                        raw[e >> 1] = (raw[e >> 1] & (0xffff0000u >> ((e & 1) * 16))) | (b << ((e & 1) * 16));
                }
            }
            if (ok != full) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    if ((ok >> e) & 1u) continue;
                    if (DT == 0)
                        raw[e & 3] = neg_inf_bits<DT>();
                    else
                        raw[e >> 1] = (raw[e >> 1] & (0xffff0000u >> ((e & 1) * 16))) | (neg_inf_bits<DT>() << ((e & 1) * 16));
                }
            }
            if (in_place && !hit && ok == full) continue;
            if (VEC) {
                *reinterpret_cast<uint4*>(dst + (size_t)e0 * Geo<DT>::kBytes) = make_uint4(raw[0], raw[1], raw[2], raw[3]);
            } else {
                for (int e = 0; e < cnt; ++e) {
                    if (DT == 0)
                        reinterpret_cast<uint32_t*>(dst)[e0 + e] = raw[e];
                    else
                        reinterpret_cast<uint16_t*>(dst)[e0 + e] = (uint16_t)(raw[e >> 1] >> ((e & 1) * 16));
                }
            }
        }
        __syncwarp();
    }
}

cudaError_t launch_logits(const LogitsParams& p, int dtype, cudaStream_t st) {
    const dim3 grid((p.V + kSlice - 1) / kSlice, p.n.S);
    if (dtype == 0) {
        if (p.vec)
            logits_kernel<0, true><<<grid, kLogThreads, 0, st>>>(p);
        else
            logits_kernel<0, false><<<grid, kLogThreads, 0, st>>>(p);
    } else {
        if (p.vec)
            logits_kernel<1, true><<<grid, kLogThreads, 0, st>>>(p);
        else
            logits_kernel<1, false><<<grid, kLogThreads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace smcsd
