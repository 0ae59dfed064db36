// logits_process.cu -- penalties for repeated tokens, biases and grammar masks on logits.
//
// Bound by the bytes of the logits (read once, written once) and the masks. One block per sequence and slice of 2048
// tokens of the vocabulary. The slice of up to kRows of the sequence's rows is copied to shared memory asynchronously
// while the block counts the slice's tokens of the history, notes the biases and the drafted tokens and makes a list
// of the tokens that anything touches; then it works out the touched tokens of every row in place, one thread each, and
// writes the rows out through the grammar mask. 128 x 5 rows of V = 128256 in bf16 with everything given take 71 us
// (4.75 TB/s, 71 % of a copy's rate; 54 us with no history): the instructions of the counting bound it, a thread's
// eight tokens of the history in each of 63 slices. Forms that were slower: looking the touched tokens up while the
// rows stream through registers (107 us: nearly every warp meets one and goes through its arithmetic for one lane);
// changing them in global memory after a copy (77 us: a chain of loads and partial writes); runs of slices by one block
// with the next rows fetched meanwhile (84 to 110 us: fewer bytes in flight).
#include <cuda_bf16.h>

#include "serve_launch.cuh"
#include "smcsd_launch.cuh"

namespace smcsd {

constexpr int kLogThreads = 256;
constexpr int kSlice = 2048;  // tokens of a block
constexpr int kRows = 3;      // rows in shared memory at a time
// Tokens of the history that a thread reads ahead, into registers: loads in flight against what short histories do not use.
// 128 x 5 rows of V = 128256 with 2 / 4 / 8 / 16: 61.2 / 61.6 / 62.7 / 65.0 us for histories of 64 tokens, 77.1 / 75.6 / 71.4 / 73.6 of
// 2048, 110 / 109 / 106 / 101 of 8192; 128 x 1 rows with 2048 tokens 40.3 / 39.1 / 35.8 / 39.1.
constexpr int kEarly = 8;
constexpr int kListed = 128;  // nodes whose tokens lie in the slice that are noted; more are looked up again

template <int DT>
struct LogShared {
    __align__(16) unsigned char rows[kRows][kSlice * Geo<DT>::kBytes];
    __align__(16) uint32_t allow[kRows][kSlice / 32];
    __align__(16) int count[kSlice];
    __align__(16) int bias[kSlice];  // 1 + index of the last bias entry of a token; then its value, if a thread has each
    uint32_t hit[kSlice / 32];       // tokens that history, bias or a node touches
    uint16_t tok[kSlice];            // the same as a list
    int2 list[kListed];              // (node, token - lo)
    int nodes, toks;                 // nodes whose tokens lie in the slice; tokens listed
};

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kLogThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
    constexpr int kE = Geo<DT>::kPerVec, kVec = kSlice / kE / kLogThreads;  // vectors of a thread in each row
    constexpr uint32_t kFull = (1u << kE) - 1u;
    static_assert(kRows * (kSlice / 32) <= kLogThreads, "a word of the mask for each thread");
    extern __shared__ __align__(16) unsigned char dyn[];
    LogShared<DT>& sh = *reinterpret_cast<LogShared<DT>*>(dyn);
    const int tid = threadIdx.x, s = blockIdx.y, lo = blockIdx.x * kSlice, len = min(kSlice, p.V - lo);
    int first;
    const int n = nodes_of(p.n, s, first, p.ws);
    if (n == 0) return;
    const bool in_place = p.out == p.logits;
    // groups of rows, all alike but the last
    const int groups = (n + kRows - 1) / kRows, per = (n + groups - 1) / groups;

    // a group of rows on its way to shared memory
    auto load = [&](int g) {
        const int t0 = g * per, rows = min(per, n - t0);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            const char* src = static_cast<const char*>(p.logits) + ((long long)(first + t0 + r) * p.V + lo) * Geo<DT>::kBytes;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int e0 = (i * kLogThreads + tid) * kE;
                if (e0 >= len) continue;
                if (ALIGNED) {
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(sh.rows[r] + e0 * Geo<DT>::kBytes);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + e0 * Geo<DT>::kBytes) : "memory");
                } else {
                    for (int e = e0; e < min(e0 + kE, len); ++e) {
                        if (DT == 0)
                            reinterpret_cast<uint32_t*>(sh.rows[r])[e] = reinterpret_cast<const uint32_t*>(src)[e];
                        else
                            reinterpret_cast<uint16_t*>(sh.rows[r])[e] = reinterpret_cast<const uint16_t*>(src)[e];
                    }
                }
            }
        }
        if (p.allowed) {
            const int r = tid / (kSlice / 32), w = tid - r * (kSlice / 32);
            if (r < rows && 32 * w < len) {
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(&sh.allow[r][w]);
                const uint32_t* src = p.allowed + (long long)(first + t0 + r) * p.allowed_words + lo / 32 + w;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
            }
        }
    };
    load(0);

    // what touches the sequence's rows
    int h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    if (p.hist_tokens) {
        h0 = __ldg(p.hist_offsets + s), h1 = __ldg(p.hist_offsets + s + 1);
        if (h0 < 0 || h1 < h0 || h1 > p.n_hist) raise_error(p.ws, kErrRange), h1 = h0 = 0;
    }
    if (p.bias_tokens) {
        b0 = __ldg(p.bias_offsets + s), b1 = __ldg(p.bias_offsets + s + 1);
        if (b0 < 0 || b1 < b0 || b1 > p.n_bias) raise_error(p.ws, kErrRange), b1 = b0 = 0;
    }
    const float rep = p.repetition ? __ldg(p.repetition + s) : 1.0f;
    const float pres = p.presence ? __ldg(p.presence + s) : 0.0f;
    const float freq = p.frequency ? __ldg(p.frequency + s) : 0.0f;
    int hist[kEarly];
#pragma unroll
    for (int x = 0; x < kEarly; ++x) hist[x] = h0 + tid + x * kLogThreads < h1 ? __ldg(p.hist_tokens + h0 + tid + x * kLogThreads) : -1;
    const int my_bias = b0 + tid < b1 ? __ldg(p.bias_tokens + b0 + tid) : -1;
    const float my_value = b0 + tid < b1 ? __ldg(p.bias_values + b0 + tid) : 0.0f;
    const int my_node = p.node_tokens && tid < n ? __ldg(p.node_tokens + first + tid) : -1;
    if (blockIdx.x == 0) {  // tokens outside the vocabulary are reported by one block
        auto inside = [&](int tok) {
            if (tok < -1 || tok >= p.V) raise_error(p.ws, kErrRange);
        };
        for (int i = h0 + tid; i < h1; i += kLogThreads) inside(__ldg(p.hist_tokens + i));
        for (int i = b0 + tid; i < b1; i += kLogThreads) inside(__ldg(p.bias_tokens + i));
        for (int i = tid; p.node_tokens && i < n; i += kLogThreads) inside(__ldg(p.node_tokens + first + i));
    }

    for (int i = tid; i < kSlice / 4; i += kLogThreads) reinterpret_cast<int4*>(sh.count)[i] = make_int4(0, 0, 0, 0);
    if (b1 > b0)
        for (int i = tid; i < kSlice / 4; i += kLogThreads) reinterpret_cast<int4*>(sh.bias)[i] = make_int4(0, 0, 0, 0);
    if (tid < kSlice / 32) sh.hit[tid] = 0;
    if (tid == 0) sh.nodes = sh.toks = 0;
    __syncthreads();
    // whether a token lies in the slice, and then marks it
    auto touch = [&](int tok, unsigned& k) {
        k = (unsigned)(tok - lo);
        if (k >= (unsigned)len) return false;
        atomicOr(&sh.hit[k >> 5], 1u << (k & 31));
        return true;
    };
    unsigned k;
#pragma unroll
    for (int x = 0; x < kEarly; ++x)
        if (touch(hist[x], k)) atomicAdd(&sh.count[k], 1);
#pragma unroll 4
    for (int i = h0 + tid + kEarly * kLogThreads; i < h1; i += kLogThreads)
        if (touch(__ldg(p.hist_tokens + i), k)) atomicAdd(&sh.count[k], 1);
    if (touch(my_bias, k)) atomicMax(&sh.bias[k], tid + 1);
    for (int i = b0 + tid + kLogThreads; i < b1; i += kLogThreads)
        if (touch(__ldg(p.bias_tokens + i), k)) atomicMax(&sh.bias[k], i - b0 + 1);
    auto note = [&](int node, int tok) {
        if (!touch(tok, k)) return;
        const int at = atomicAdd(&sh.nodes, 1);
        if (at < kListed) sh.list[at] = make_int2(node, (int)k);
    };
    note(tid, my_node);
    for (int i = tid + kLogThreads; p.node_tokens && i < n; i += kLogThreads) note(i, __ldg(p.node_tokens + first + i));
    __syncthreads();
    if (tid < kSlice / 32) {
        uint32_t left = sh.hit[tid];
        if (left)
            for (int at = atomicAdd(&sh.toks, __popc(left)); left; left &= left - 1) sh.tok[at++] = (uint16_t)(32 * tid + __ffs(left) - 1);
    }
    // with one entry a thread, the entries that count put their values in place of their numbers
    const bool few = b1 - b0 <= kLogThreads;
    if (few && b1 > b0) {
        k = (unsigned)(my_bias - lo);
        const bool counts = k < (unsigned)len && sh.bias[k] == tid + 1;
        __syncthreads();
        if (counts) sh.bias[k] = __float_as_int(my_value);
    }

    for (int g = 0; g < groups; ++g) {
        const int t0 = g * per, rows = min(per, n - t0);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        const int nodes = sh.nodes, toks = sh.toks;
        const bool listed = nodes <= kListed;
        for (int i = tid; i < toks * rows; i += kLogThreads) {
            const int r = i / toks, c = sh.tok[i - r * toks], t = t0 + r;
            int count = sh.count[c];
            for (int x = 0; x < (listed ? nodes : n); ++x) {
                const int2 e = listed ? sh.list[x] : make_int2(x, __ldg(p.node_tokens + first + x) - lo);
                if (e.y != c) continue;
                count += p.mask ? (__ldg(p.mask + (long long)(first + t) * p.words + (e.x >> 5)) >> (e.x & 31)) & 1u : e.x <= t;
            }
            unsigned char* row = sh.rows[r];
            float z;
            if (DT == 0)
                z = reinterpret_cast<const float*>(row)[c];
            else
                z = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c]);
            if (count > 0) {
                z = z > 0.0f ? z / rep : z * rep;
                z = z - freq * (float)count;
                z = z - pres;
            }
            if (b1 > b0) {
                const int x = sh.bias[c];
                if (x) z = z + (few ? __int_as_float(x) : __ldg(p.bias_values + b0 + x - 1));
            }
            if (DT == 0)
                reinterpret_cast<float*>(row)[c] = z;
            else
                reinterpret_cast<__nv_bfloat16*>(row)[c] = __float2bfloat16_rn(z);
        }
        if (toks > 0) __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            char* dst = static_cast<char*>(p.out) + ((long long)(first + t0 + r) * p.V + lo) * Geo<DT>::kBytes;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int e0 = (i * kLogThreads + tid) * kE;
                if (e0 >= len) continue;
                const uint32_t allow = p.allowed ? (sh.allow[r][e0 >> 5] >> (e0 & 31)) & kFull : kFull;
                if (in_place && allow == kFull && !((sh.hit[e0 >> 5] >> (e0 & 31)) & kFull)) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(sh.rows[r] + e0 * Geo<DT>::kBytes);
                uint32_t raw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (DT == 0) {
                        if (!((allow >> x) & 1u)) raw[x] = neg_inf_bits<DT>();
                    } else {
                        // bits 2 x and 2 x + 1 select the halves that are let through
                        const uint32_t keep =
                            ((allow >> (2 * x)) & 1u ? 0xffffu : 0u) | ((allow >> (2 * x)) & 2u ? 0xffff0000u : 0u);
                        raw[x] = (raw[x] & keep) | (0xff80ff80u & ~keep);
                    }
                }
                if (ALIGNED) {
                    __stcs(reinterpret_cast<uint4*>(dst + e0 * Geo<DT>::kBytes), make_uint4(raw[0], raw[1], raw[2], raw[3]));
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        if (e >= len - e0) break;
                        if (DT == 0)
                            reinterpret_cast<uint32_t*>(dst)[e0 + e] = raw[e & 3];
                        else
                            reinterpret_cast<uint16_t*>(dst)[e0 + e] = (uint16_t)(raw[(e >> 1) & 3] >> ((e & 1) * 16));
                    }
                }
            }
        }
        if (g + 1 < groups) {
            __syncthreads();
            load(g + 1);
        }
    }
}

template <int DT, bool ALIGNED>
static cudaError_t launch_logits_t(const LogitsParams& p, cudaStream_t st) {
    auto kern = logits_kernel<DT, ALIGNED>;
    constexpr int smem = sizeof(LogShared<DT>);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3((p.V + kSlice - 1) / kSlice, p.n.S), kLogThreads, smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_logits(const LogitsParams& p, int dtype, cudaStream_t st) {
    if (dtype == 0) return p.vec ? launch_logits_t<0, true>(p, st) : launch_logits_t<0, false>(p, st);
    return p.vec ? launch_logits_t<1, true>(p, st) : launch_logits_t<1, false>(p, st);
}

}  // namespace smcsd
