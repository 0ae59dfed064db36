// attn_tc.cuh -- what the two tensor-core kernels of tree_attention share: tcgen05 / TMA / mbarrier
// instructions, bounded waits, the pieces of a block's share handed round, the warps that bring the pages of keys
// and values into their rings, the masks of a tile's positions, and the tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_plan.cuh"

namespace smcsd {

namespace {

constexpr int kTile = 128;        // keys of a tile

// ---- instructions ----

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(2000u)  // at most about 2 us
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// One thread of a converged warp, the same each time. Work that is issued by one thread stays in code that the whole
// warp runs up to the instruction itself, with values that are the same in all lanes (uniform): the instructions
// of the tensor core and the copy engine take their operands from the warp's uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int group, int page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(group), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// both operands in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// the first operand in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void ld32(uint32_t addr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) { return attn_ex2(x); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Tiles in shared memory: 128-byte swizzle, blocks of 8 rows x 64 columns (1 KB) with a row's D / 64 blocks side by
// side: [row / 8][column / 64][row % 8][column % 64]. One copy brings a page in this order.
template <int D>
struct TileGeo {
    static constexpr int kHalves = D / 64;
    static constexpr int kGroup = kHalves * 1024;  // bytes of 8 rows
    static constexpr int kBytes = 16 * kGroup;     // of 128 rows
    // row r, 16-byte chunk ch (of D / 8) of a row
    static __host__ __device__ constexpr int at(int r, int ch) {
        return (r >> 3) * kGroup + (ch >> 3) * 1024 + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4);
    }
    // 16 columns of the sum's dimension (rows along the sum): step k
    static __host__ __device__ constexpr int step(int k) { return (k >> 2) * 1024 + (k & 3) * 32; }
};

// Shared-memory operand of a product. `next8` bytes from one group of 8 rows to the next; where the rows lie along the
// sum (values: a key's columns in a row), `block` bytes from one block of 64 columns to the next.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t next8, uint32_t block) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(next8 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// Instruction: float32 sums, bf16 operands, 128 x n outputs; amn / bmn: that operand's rows lie along the output
__host__ __device__ constexpr uint32_t instruction(int n, int amn, int bmn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16) | ((uint32_t)(n / 8) << 17) |
           ((128u / 16) << 24);
}

struct Ctl {
    void* ws;
    int* abort;
};
// Waits are bounded: each try suspends the thread for a few microseconds at most, and after kTries of them (0.1 to
// a few seconds) every later wait of the block returns; the error is recorded at the block's end.
constexpr int kTries = 1 << 19;
// one thread of a warp
__device__ __forceinline__ void wait1(const Ctl& c, uint32_t bar, uint32_t parity) {
    int tries = 0;
#pragma unroll 1
    while (!mbar_try(bar, parity)) {
        if (++tries < kTries && !*reinterpret_cast<volatile int*>(c.abort)) continue;
        *reinterpret_cast<volatile int*>(c.abort) = 1;
        break;
    }
}
// a whole warp
__device__ __forceinline__ void wait(const Ctl& c, uint32_t bar, uint32_t parity) {
    wait1(c, bar, parity);
    __syncwarp();
}

// The pieces of a block's share as one warp hands them to the others. They stay in shared memory, where each reader takes from
// them what it needs when it needs it (copies of its own were spilled, and with nearly all of the SM's memory in use as shared
// memory a spilled value comes from the second-level cache), and reports when it is through with one.
constexpr int kPieces = 8;
struct PieceRing {
    PieceInfo piece[kPieces];
    PieceInfo pending[2];  // cut units' pieces, to be reported at the end
    uint64_t full[kPieces], empty[kPieces];
    int last[2];
    __device__ __forceinline__ void init(int readers) {
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), readers);
        }
    }
    // one warp
    __device__ __forceinline__ void put(const Ctl& ctl, uint32_t i, const PieceInfo& c, int lane) {
        if (i >= kPieces) wait(ctl, smem_u32(&empty[i % kPieces]), (i / kPieces - 1) & 1);
        if (lane == 0) {
            piece[i % kPieces] = c;
            mbar_arrive(smem_u32(&full[i % kPieces]));
        }
        __syncwarp();
    }
    // Waits for the i-th piece; its rows (none after a wait that ran out).
    __device__ __forceinline__ int get(const Ctl& ctl, uint32_t i) const {
        wait(ctl, smem_u32(&full[i % kPieces]), (i / kPieces) & 1);
        return uniform(*reinterpret_cast<volatile int*>(ctl.abort) ? 0 : piece[i % kPieces].rows);
    }
    __device__ __forceinline__ const PieceInfo& at(uint32_t i) const { return piece[i % kPieces]; }
    __device__ __forceinline__ void done(uint32_t i) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&empty[i % kPieces]));
        __syncwarp();
    }
};

// After a wait that ran out: records the error, and gives copies and products in flight time to land before the block's
// shared and tensor memory is handed on.
__device__ __forceinline__ void settle(const Ctl& c) {
    if (!*reinterpret_cast<volatile int*>(c.abort)) return;
    raise_timeout(c.ws);
    const unsigned long long t0 = now_ns();
    while (now_ns() - t0 < 20000000ull) __nanosleep(1000);
}
// the warps of the softmax
template <int kThreads>
__device__ __forceinline__ void rows_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
// Whether any thread of them says yes.
template <int kThreads>
__device__ __forceinline__ bool rows_any(bool yes) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)yes), "n"(kThreads)
                 : "memory");
    return r != 0;
}

// ---- keys and values ----

// A ring of shared-memory stages that one warp fills, tile after tile.
template <int kStages>
struct Ring {
    uint64_t full[kStages], empty[kStages];
    __device__ __forceinline__ void init(int readers) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), readers);
        }
    }
};

// Fills a ring with the pages of a run of tiles (one warp; one for the keys and one for the values). A lane holds one
// page id (a box: up to 128 positions of one page); 32 ids are read at a time, the next 32 while these are used. The
// copies are issued by one thread with the ids handed round four at a time: lanes issuing a copy each take turns
// anyway, at four times the cost. Pages past the end are not read.
template <int D>
struct Filler {
    using T = TileGeo<D>;
    const CUtensorMap* map;
    uint64_t *full, *empty;
    uint32_t stages, ring, st, round;
    __device__ __forceinline__ Filler(const CUtensorMap* m, uint64_t* f, uint64_t* e, int n, uint32_t addr)
        : map(m), full(f), empty(e), stages(n), ring(addr), st(0), round(0) {}
    // A lane's page id among the 32 boxes of a piece from 32 * batch on.
    __device__ __forceinline__ int page_id(const AttnParams& p, const PieceInfo& c, int batch, int lane) {
        const int at = (32 * batch + lane) << min(p.page_shift, 7);
        return at < min(c.n * kTile, c.end - c.key0) ? __ldg(p.table + (long long)c.seq * p.pages_per_seq + ((c.key0 + at) >> p.page_shift)) : 0;
    }
    __device__ __forceinline__ int checked(const AttnParams& p, int id) {
        if (id < 0 || id >= p.num_pages) {
            raise_error(p.ws, kErrRange);
            id = 0;
        }
        return id;
    }
    // the tiles of a piece, whose first 32 ids were read before; false after a wait that ran out
    __device__ __forceinline__ bool fill(const AttnParams& p, const Ctl& ctl, const PieceInfo& c, int id, int lane) {
        const int hkv = c.hkv, n = c.n, key0 = c.key0;
        const int box_shift = min(p.page_shift, 7), box = 1 << box_shift, nbox = kTile >> box_shift;
        const int last = min(n * kTile, c.end - key0);  // end of the positions
        const int bytes = box * D * 2;
        int next = page_id(p, c, 1, lane), batch = 1;
        id = checked(p, id);
#pragma unroll 1
        for (int t = 0, x = 0; t < n; ++t, x += nbox) {
            if (x == 32) {
                x = 0;
                id = checked(p, next);
                next = page_id(p, c, ++batch, lane);
            }
            wait(ctl, smem_u32(&empty[st]), (round & 1) ^ 1);  // at once the first time round
            if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(ctl.abort))) return false;
            const int ust = uniform(st), boxes = uniform(min(nbox, (last - t * kTile + box - 1) >> box_shift));
            const uint32_t bar = smem_u32(&full[ust]);
            uint32_t to = ring + ust * T::kBytes;
            const int at = uniform((hkv * p.page_size + ((key0 + t * kTile) & (p.page_size - 1))) >> 3);
            if (elect_one()) mbar_expect_tx(bar, (uint32_t)(boxes * bytes));
            __syncwarp();
#pragma unroll 1
            for (int b = 0; b < boxes; b += 4, to += 4 * bytes) {
                int page[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) page[y] = __shfl_sync(0xffffffffu, id, (x + b + y) & 31);
                if (elect_one()) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (b + y < boxes) tma_page(to + y * bytes, map, at, page[y], bar);
                }
            }
            if (++st == stages) st = 0, ++round;
        }
        return true;
    }
};

// ---- masks ----

// Keys of a tile that the product with V takes, of `keys` that it has: up to the next 16 (one step of it).
__device__ __forceinline__ int tile_steps(int keys) { return (min(keys, kTile) + 15) >> 4; }

// Zeroes what the product with V must not meet in a tile of `keys` keys: in what it takes of the rows past the end everything,
// in those of the nodes (from `first` on) NaN and infinities, which rows of zero weight would turn into NaN. Thread i of n takes
// every n-th 16 bytes; true if it found some.
template <int D>
__device__ __forceinline__ bool clean_values(uint32_t tile, int first, int keys, int i, int n) {
    auto at = [&](int x) {
        const int r = x / (D / 8), ch = x % (D / 8);
        return tile + (r >> 3) * TileGeo<D>::kGroup + (ch >> 3) * 1024 + (r & 7) * 128 + (ch & 7) * 16;
    };
    const int nodes = min(keys, kTile) * (D / 8), end = 16 * tile_steps(keys) * (D / 8);
    bool found = false;
#pragma unroll 1
    for (int x = first * (D / 8) + i; x < nodes; x += 2 * n) {
        uint32_t v[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y)  // the last one twice rather than none
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[y][0]), "=r"(v[y][1]), "=r"(v[y][2]), "=r"(v[y][3])
                         : "r"(at(x + y * n < nodes ? x + y * n : x))
                         : "memory");
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((v[y][e] & 0x7f80u) == 0x7f80u) v[y][e] &= 0xffff0000u, bad = true;
                if ((v[y][e] & 0x7f800000u) == 0x7f800000u) v[y][e] &= 0x0000ffffu, bad = true;
            }
            if (!bad) continue;
            found = true;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at(x + y * n < nodes ? x + y * n : x)), "r"(v[y][0]), "r"(v[y][1]),
                         "r"(v[y][2]), "r"(v[y][3])
                         : "memory");
        }
    }
#pragma unroll 1
    for (int x = nodes + i; x < end; x += n) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at(x)), "r"(0) : "memory");
    return found;
}

// Which of 32 positions from `base` on a row sees.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
__device__ __forceinline__ uint32_t seen32(const AttnParams& p, const uint32_t* mask_row, int node, int ctx, int keys, int base) {
    const int j0 = base - ctx;
    uint32_t nodes;
    if (mask_row) {
        const int wd = j0 >> 5, sh = j0 & 31;  // floor
        const uint32_t lo = wd >= 0 && wd < p.words ? __ldg(mask_row + wd) : 0u;
        const uint32_t hi = wd + 1 >= 0 && wd + 1 < p.words ? __ldg(mask_row + wd + 1) : 0u;
        nodes = __funnelshift_r(lo, hi, sh);
    } else {
        nodes = low_bits(node + 1 - j0);
    }
    return (low_bits(-j0) | nodes) & low_bits(keys - base);
}

// ---- tensor maps ----

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A cache as [num_pages][Hkv * page_size / 8][8][D / 64][64], taken with the blocks of 64 columns outside the 8 rows: a
// box is one page of one head (or 128 positions of it) in the order of TileGeo.
bool encode_cache(CUtensorMap* m, const void* base, const AttnParams& p) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row = (cuuint64_t)p.D * 2, halves = (cuuint64_t)p.D / 64;
    const cuuint64_t dim[5] = {64, 8, halves, (cuuint64_t)p.Hkv * p.page_size / 8, (cuuint64_t)p.num_pages};
    const cuuint64_t stride[4] = {row, 128, 8 * row, row * p.Hkv * p.page_size};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, (cuuint32_t)(p.page_size < kTile ? p.page_size : kTile) / 8, 1},
                     one[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Kernel>
cudaError_t launch_tc(Kernel kern, int threads, int smem, const AttnParams& p, cudaStream_t st) {
    CUtensorMap mk, mv;
    if (!encode_cache(&mk, p.k_cache, p) || !encode_cache(&mv, p.v_cache, p)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ncta_max);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.planned ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, mk, mv);
}

}  // namespace

}  // namespace smcsd
