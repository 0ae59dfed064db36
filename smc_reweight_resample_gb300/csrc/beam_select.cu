// beam_select.cu -- the best continuations of every group's beams over the vocabulary.
//
// Candidate (beam i, token v) of a group has the score s_i + c z_iv - L_i with L_i = log sum_v exp(c z_iv), c = 1 / temperature; with
// the row's maximum m_i that is s_i + c (z_iv - m_i) - log S_i, S_i = sum_v exp(c (z_iv - m_i)). The M best of a group's N * V
// candidates are wanted, in the order of score, beam, token.
//
// One pass over the logits: a warp takes a chunk of 4 KB (eight 16-byte vectors a lane, loads back to back) and leaves its
// maximum, its sum of exp(c (z - maximum)) and the maxima of its sixteen sets (a set: the vectors of half the lanes of one load,
// 256 contiguous bytes). Nothing is selected on the way. Of ranges of tokens ordered by their maxima, ties by place, the first M
// hold the M best tokens: each of these M ranges has a token that comes before any token of a range behind them. So the last
// block of a group to finish
//   - adds up the beams' sums, which gives every score up to the beam's own constant,
//   - finds the M (to 5/4 M + 8) best of the group's sets, where there are many of its chunks first and then of their sets, by
//     bisection on their maxima's scores,
//   - reads these sets again and keeps what is not below the last of them: a little more than M candidates,
//   - ranks them by counting.
// Scores are compared as double-floats (FP64 runs at two lanes a clock here). Of one beam this
// order is exact, whatever its sum; between beams it is as good as the sums and their logarithms (kTol). Where two scores of different beams that decide
// anything are nearer than that, the block computes these beams' sums again to 2e-10 and selects anew.
//
// A row alone (groups of one) is selected by its logits, without its sum: less code, 64 registers, eight blocks of four warps in an SM.
// The 64 best of 2048 rows of 128256 bf16 take 124 us, the one best 106; reading alone 93, and 78 at the copy rate: what is left
// is the selection of the last blocks and the four warps that each block selects with. 8 groups of 16 beams of 128256, 12 of them read,
// take 20 us: 6 for the reading (25 MB), 1.3 for the blocks' meeting, 1.6 for the sums, 5.6 for the two levels, 0.6 for the sets, 2.2
// for the order, 2 for the launch: latency. The sums of doubtful beams cost 30 us for a row of 128256.
#include "f32x2.cuh"
#include "ops_launch.cuh"
#include "smcsd_launch.cuh"

namespace smcsd {

// Blocks of 512 threads for few groups, whose rows several blocks share; of 128 for many groups (a block each), so that one
// group's selection, which is latency, goes on beside the reading of others.
constexpr int kBeamWide = 512, kBeamNarrow = 128;
constexpr int kBeamMostCands = 1024;  // candidates that are ranked

// How far the scores of two beams may be off from one another with hardware exponentials. A sum, relative: the exponential 2^-22; its
// argument's roundings (of z - m, of c log2 e and of their product: 2.5 * 2^-24 of it, and it is 31 on the average at most, the
// distribution's entropy over up to 2^31 tokens), times ln 2: 3.2e-6; 8 + 3 + 1 + 5 additions one after another and 8 + 5 of
// chunks, 2^-24 each; the chunks' scale 2^-22; the logarithm 4e-8: 6.1e-6. Two of them: 1.2e-5.
constexpr float kTol = 1.25e-5f;

// A score as an unsigned integer of the same order: the high float first, then the low one (of a normalised double-float). 0 is
// no score: minus infinity, and NaN, which double-floats make of what lies below float32's range (tokens masked with the lowest
// value, by a temperature below 1).
__device__ __forceinline__ uint32_t float_order(float f) {
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of_order(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(dd s) {
    if (!(s.hi > kNegInf) || !(s.hi < kPosInf)) return 0;
    return (uint64_t)float_order(s.hi + 0.0f) << 32 | float_order(s.lo + 0.0f);  // -0 is 0
}
__device__ __forceinline__ dd key_value(uint64_t k) { return dd{float_of_order((uint32_t)(k >> 32)), float_of_order((uint32_t)k)}; }
// c (z - m) + base, m being the row's maximum
__device__ __forceinline__ uint64_t score_key(const BeamParams& p, float z, float m, float2 base) {
    if (!(z > kNegInf)) return 0;
    return key_of(dd_add(dd_mul(two_sum(z, -m), dd{p.c_hi, p.c_lo}), dd{base.x, base.y}));
}

// Row r: its first vector begins `shift` elements before the row, at a multiple of 16 bytes.
template <int DT>
struct BeamRow {
    const char* at;  // first vector
    const char* row;
    int shift, V;
};
template <int DT>
__device__ __forceinline__ BeamRow<DT> beam_row(const BeamParams& p, long long r) {
    BeamRow<DT> b;
    b.row = static_cast<const char*>(after_wait(p.logits)) + r * p.row_stride * Geo<DT>::kBytes;
    const int off = (int)(reinterpret_cast<uintptr_t>(b.row) & 15u);
    b.at = b.row - off;
    b.shift = off / Geo<DT>::kBytes;
    b.V = p.V;
    return b;
}
__device__ __forceinline__ uint4 ld_vec(const char* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// Vector v of the row; tokens outside the row are -inf, and memory outside the row is not read.
template <int DT>
__device__ __forceinline__ uint4 beam_vec(const BeamRow<DT>& b, int v) {
    constexpr int PV = Geo<DT>::kPerVec;
    const long long e0 = (long long)v * PV - b.shift;
    if (e0 >= 0 && e0 + PV <= b.V) return ld_vec(b.at + 16ll * v);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = DT == 0 ? neg_inf_bits<0>() : neg_inf_bits<1>() * 0x10001u;
        if (DT == 0) {
            if (e0 + i >= 0 && e0 + i < b.V) w[i] = logit_bits<0>(b.row, e0 + i);
        } else {
            const long long e = e0 + 2 * i;
            if (e >= 0 && e < b.V) w[i] = (w[i] & 0xffff0000u) | logit_bits<1>(b.row, e);
            if (e + 1 >= 0 && e + 1 < b.V) w[i] = (w[i] & 0xffffu) | logit_bits<1>(b.row, e + 1) << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ void unpack(const uint4& x, float* f) {
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
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& x) {
    if (DT == 0)
        return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
    const uint32_t m = max_bf16x2(max_bf16x2(x.x, x.y), max_bf16x2(x.z, x.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
}

// Maximum over the lanes of a mask, which all of them give.
__device__ __forceinline__ float part_max(float v, unsigned mask) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(mask));
    return r;
}

// One chunk of a row: its maximum, sum and set maxima. NaN and +inf show in the sum.
template <int DT>
__device__ __forceinline__ void beam_chunk(const BeamParams& p, const BeamRow<DT>& b, int chunk, float* maximum, float* total, float* sets, int lane) {
    constexpr int PV = Geo<DT>::kPerVec;
    constexpr int kLoads = kBeamSets / 2;
    uint4 x[kLoads];
    const int v0 = chunk * kLoads * 32;
    const long long e0 = (long long)v0 * PV - b.shift;
    if (e0 >= 0 && e0 + kLoads * 32 * PV <= b.V) {
#pragma unroll
        for (int s = 0; s < kLoads; ++s) x[s] = ld_vec(b.at + 16ll * (v0 + s * 32 + lane));
    } else {
#pragma unroll
        for (int s = 0; s < kLoads; ++s) x[s] = beam_vec<DT>(b, v0 + s * 32 + lane);
    }
    float m = kNegInf, mine = kNegInf;
    const unsigned half = lane < 16 ? 0xffffu : 0xffff0000u;
#pragma unroll
    for (int s = 0; s < kLoads; ++s) {
        const float a = part_max(vec_max<DT>(x[s]), half);
        if ((lane & 15) == s) mine = a;
        m = fmaxf(m, a);
    }
    m = warp_max(m);
    float sum = 0.0f;
    if (m > kNegInf) {
        const f32x2 m2 = pair(-m, -m), c2 = pair(p.c2, p.c2);
        f32x2 sums[Vec<DT>::kPairs];
#pragma unroll
        for (int k = 0; k < Vec<DT>::kPairs; ++k) sums[k] = pair(0.0f, 0.0f);
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
            const Vec<DT> v(x[s]);
#pragma unroll
            for (int k = 0; k < Vec<DT>::kPairs; ++k) sums[k] = add2(sums[k], exp2_2(mul2(add2(v.x[k], m2), c2)));
        }
#pragma unroll
        for (int k = 1; k < Vec<DT>::kPairs; ++k) sums[0] = add2(sums[0], sums[k]);
        float lo, hi;
        halves(sums[0], lo, hi);
        sum = warp_sum(lo + hi);
    } else {
        // nothing but -inf, unless there are NaN, which the maxima pass over
        bool nan = false;
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
            float f[PV];
            unpack<DT>(x[s], f);
#pragma unroll
            for (int i = 0; i < PV; ++i) nan |= f[i] != f[i];
        }
        if (__any_sync(0xffffffffu, nan)) sum = __int_as_float(0x7fffffff);
    }
    if ((lane & 15) < kLoads) sets[2 * (lane & 15) + (lane >> 4)] = mine;
    if (lane == 0) *maximum = m, *total = sum;
}

// A block's shared memory, sized by the call, by offsets (which keep its accesses in 32 bits).
extern __shared__ __align__(16) char s_beam[];
struct BeamShared {
    int N, most, M, cands;
    template <typename T>
    __device__ __forceinline__ T* at_offset(int bytes) const {
        return reinterpret_cast<T*>(s_beam + bytes);
    }
    __device__ __forceinline__ float2& base(int i) const { return at_offset<float2>(0)[i]; }  // [N] s_i - log S_i, the beam's best score (of a finished beam s_i)
    __device__ __forceinline__ float& zmax(int i) const { return at_offset<float>(8 * N)[i]; }   // [N] the row's maximum
    __device__ __forceinline__ float& zmin(int i) const { return at_offset<float>(12 * N)[i]; }   // [N] no candidate below this logit
    __device__ __forceinline__ int& live(int i) const { return at_offset<int>(16 * N)[i]; }       // [N] beams whose rows are read
    __device__ __forceinline__ int& over(int i) const { return at_offset<int>(20 * N)[i]; }       // [N] finished beams
    __device__ __forceinline__ int* list1() const { return at_offset<int>(24 * N); }              // [most] chunks
    __device__ __forceinline__ int* list2() const { return at_offset<int>(24 * N + 4 * most); }   // [most] sets
    __device__ __forceinline__ int& order(int i) const { return at_offset<int>(24 * N + 8 * most)[i]; }  // [M + 1]
    __device__ __forceinline__ int& unsure(int i) const { return at_offset<int>(24 * N + 8 * most + 4 * (M + 1))[i]; }  // [N] beams in doubt
    __host__ __device__ __forceinline__ int tail() const { return (28 * N + 8 * most + 4 * (M + 1) + 15) & ~15; }
    __device__ __forceinline__ float& score(int i) const { return at_offset<float>(tail())[i]; }  // [keys] maxima, then their scores; shares its
                                                                                                 // memory with the candidates
    __device__ __forceinline__ uint64_t& key(int i) const { return at_offset<uint64_t>(tail())[i]; }             // [cands + N]
    __device__ __forceinline__ uint64_t& at(int i) const { return at_offset<uint64_t>(tail())[cands + N + i]; }  // [cands + N] beam, token
};
struct BeamCounts {
    int nlive, nover, count, last;
    int chunks, narrowed;  // chunks in list1; whether candidates were left out
    unsigned votes[3][2];
    unsigned best;  // the best beam's score, by float_order (0: there is none)
    unsigned long long reduce;
    dd part[kBeamWide / 32];
};
__host__ __device__ inline BeamShared beam_shared(int N, int M) {
    return BeamShared{N, M + M / 4 + 8, M, 4 * M + 64 < kBeamMostCands ? 4 * M + 64 : kBeamMostCands};
}
// Scores of a level: of the sets of all chunks kept, and of all chunks; of all sets where those are not many more.
__host__ __device__ inline int beam_keys(const BeamShared& s, int chunks, int threads) {
    int n = kBeamSets * s.most;
    const int some = threads == kBeamWide ? 8192 : 2048;
    if (n < some) n = some;
    return n < chunks ? chunks : n;
}
inline size_t beam_shared_bytes(int N, int M, int chunks, int threads) {
    const BeamShared s = beam_shared(N, M);
    const size_t keys = 4 * (size_t)beam_keys(s, chunks, threads), cands = 16 * (size_t)(s.cands + N);
    return (size_t)s.tail() + (keys > cands ? keys : cands);
}

constexpr float kLowest = -3.402823466e38f;

// What is kept of a level's n items: those whose key is above K, and those with K before place I.
struct Cut {
    uint64_t K;
    int I;
};
__device__ __forceinline__ bool kept(const Cut& c, uint64_t key, int i) { return key > c.K || (key == c.K && i < c.I); }

// Keys by bisection of their bits and then of their places, for levels whose scores differ too little for find_cut: between M and
// `most` of them, the first in the order of keys and places. There are more than `most`.
template <int TH, typename F>
__device__ __noinline__ Cut find_cut_exact(int n, int M, int most, F key_of) {
    const auto count = [&](uint64_t K, int I) {
        int c = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x < n; i += TH) c += __syncthreads_count(i < n && kept(Cut{K, I}, key_of(i), i));
        return c;
    };
    uint64_t lo = 1, hi = ~0ull;  // more than `most` from lo on, fewer than M from hi on
    while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        const int c = count(mid, n);
        if (c > most)
            lo = mid;
        else if (c < M)
            hi = mid;
        else
            return Cut{mid, n};
    }
    int a = 0, b = n;  // many are equal to lo: the first places of them
    while (b - a > 1) {
        const int mid = a + (b - a) / 2, c = count(lo, mid);
        if (c < M)
            a = mid;
        else if (c > most)
            b = mid;
        else
            return Cut{lo, mid};
    }
    return Cut{lo, b};
}

// A score from which on there are between M and `most` of the n scores: a bisection of values, four at a time, since the M best are
// mostly within a few nats (`unit`) of the best. Fails where ties, or scores next to the best, leave none.
template <int TH>
__device__ __forceinline__ bool find_cut(const BeamShared& s, BeamCounts& c, int n, int M, int most, float best, float unit, float& from) {
    float above = best, below = kNegInf, step = 0.5f * unit;  // the border lies between them: more than `most` from `below` on
    for (int turn = 0; turn < 16; ++turn) {
        float t[4];
        if (below == kNegInf) {
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = best - step * (float)(1 << k);
            step *= turn < 2 ? 16.0f : 65536.0f;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = above + (below - above) * (0.2f * (float)(k + 1));
        }
        unsigned lo = 0, hi = 0;  // counts of 16 bits: n is less than 65536
        for (int i = threadIdx.x; i < n; i += TH) {
            const float x = s.score(i);
            lo += (x >= t[0] ? 1u : 0u) + (x >= t[1] ? 0x10000u : 0u);
            hi += (x >= t[2] ? 1u : 0u) + (x >= t[3] ? 0x10000u : 0u);
        }
        lo = __reduce_add_sync(0xffffffffu, lo);
        hi = __reduce_add_sync(0xffffffffu, hi);
        const int slot = turn % 3;
        if ((threadIdx.x & 31) == 0 && hi) {
            atomicAdd(&c.votes[slot][0], lo);
            atomicAdd(&c.votes[slot][1], hi);
        }
        __syncthreads();
        lo = c.votes[slot][0], hi = c.votes[slot][1];
        if (threadIdx.x < 2) c.votes[(turn + 2) % 3][threadIdx.x] = 0;  // all have read that one by the last barrier
        const int got[4] = {(int)(lo & 0xffffu), (int)(lo >> 16), (int)(hi & 0xffffu), (int)(hi >> 16)};
        const float was_above = above, was_below = below;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (got[k] >= M && got[k] <= most) {
                from = t[k];
                return true;
            }
            if (got[k] < M) above = t[k];
        }
#pragma unroll
        for (int k = 3; k >= 0; --k)
            if (got[k] > most) below = t[k];
        if (!(t[3] > kNegInf) || (was_above == above && was_below == below && below != kNegInf)) break;
    }
    return false;
}
template <int TH>
__device__ __forceinline__ void clear_votes(BeamCounts& c) {
    __syncthreads();
    if (threadIdx.x < 6) c.votes[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    if (threadIdx.x == 0) c.count = 0;
    __syncthreads();
}

// Puts a short list of distinct places in ascending order.
template <int TH>
__device__ void sort_list(int* list, int n) {
    constexpr int kEach = (kBeamMost + kBeamMost / 4 + 8 + TH - 1) / TH;
    int mine[kEach], rank[kEach];
#pragma unroll
    for (int t = 0; t < kEach; ++t) {
        const int i = threadIdx.x + t * TH;
        rank[t] = 0;
        if (i < n) {
            mine[t] = list[i];
            for (int j = 0; j < n; ++j) rank[t] += list[j] < mine[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kEach; ++t)
        if ((int)threadIdx.x + t * TH < n) list[rank[t]] = mine[t];
    __syncthreads();
}

// A level: the chunks of the group's live beams; the sets of all of them where they are few; or the sets of the chunks in list1.
struct Level {
    const float* maxima;  // of the group's rows
    int cpr, n, log;      // chunks of a row, items, log2 of the items of a chunk
    bool listed;
    FastDiv chunks;       // by the chunks of a row
    // an item's live beam, by its place among them, and where its maximum stands
    __device__ __forceinline__ int chunk(const BeamShared& s, int i) const { return listed ? s.list1()[i >> log] : i >> log; }
    __device__ __forceinline__ int beam(const BeamShared& s, int i) const { return s.live((int)fast_div((uint32_t)chunk(s, i), chunks)); }
    __device__ __forceinline__ float z(const BeamShared& s, int i) const {
        const int k = chunk(s, i), l = (int)fast_div((uint32_t)k, chunks);
        return __ldcg(maxima + (((long long)s.live(l) * cpr + (k - l * cpr)) << log) + (i & ((1 << log) - 1)));
    }
};
// The first level (sets at once, where they fit) or the second (the sets of n1 chunks).
template <int TH>
__device__ __forceinline__ Level level_of(const BeamParams& p, const BeamShared& s, int g, int nlive, bool second, int n1) {
    static_assert(kBeamSets == 16, "shifts by 4");
    Level v;
    v.log = second || nlive * p.cpr <= beam_keys(s, p.N * p.cpr, TH) / kBeamSets ? 4 : 0;
    v.listed = second;
    v.cpr = p.cpr;
    v.n = (second ? n1 : nlive * p.cpr) << v.log;
    v.chunks = p.div_cpr;
    v.maxima = ws_ptr<const float>(p.ws, v.log ? p.sets : p.maxima) + ((long long)g * p.N * p.cpr << v.log);
    return v;
}
// Keys of a level's items, for what is not done as a rule.
struct LevelKey {
    const BeamParams* p;
    BeamShared s;
    Level level;
    __device__ __forceinline__ uint64_t operator()(int i) const {
        const int beam = level.beam(s, i);
        return score_key(*p, level.z(s, i), s.zmax(beam), s.base(beam));
    }
};
// An item's score: in float32, off by at most three roundings (of the difference, of the factor, of the sum) of its terms, and for one beam in the order of
// the logits; or as the high half of its key. The terms are the beam's constant b and c (z - m), which is not above 0: no larger than the score
// where b <= 0, than the score and b together where it is above 0.
constexpr float kScoreError = 3e-7f;
// How far a float32 score next to `score` may be off, by that and by the sums.
__device__ __forceinline__ float doubt_of(const BeamCounts& c, float score) {
    return kTol + 2.0f * kScoreError * (fabsf(score) + fmaxf(float_of_order(c.best), 0.0f));
}
__device__ __forceinline__ float level_score(const BeamParams& p, const BeamShared& s, const Level& level, int i, float z, bool exact) {
    const int beam = level.beam(s, i);
    if (!exact) return z > kNegInf ? fmaf(p.c_hi, z - s.zmax(beam), s.base(beam).x) : kNegInf;
    const uint64_t key = score_key(p, z, s.zmax(beam), s.base(beam));
    return key ? float_of_order((uint32_t)(key >> 32)) : kNegInf;
}

// The places of a level's n items that hold the group's M best tokens, in `list`; returns how many. All that are there, if they are
// no more than `most`. `floor`: a score, up to kScoreError; no item below it has been kept.
template <int TH, typename F>
__device__ __forceinline__ int choose(const BeamShared& s, BeamCounts& c, int n, float best, float unit, const F& key_of, int* list, float& floor,
                                      bool& by_place) {
    const int most = s.most;
    float from = kLowest;
    Cut cut{0, n};
    by_place = false;
    clear_votes<TH>(c);
    bool ok = n <= most;
    if (!ok) {
        ok = find_cut<TH>(s, c, n, s.M, most, best, unit, from);
        if (!ok) {
            int some = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x < n; i += TH) some += __syncthreads_count(i < n && s.score(i) > kNegInf);
            ok = some <= most;  // fewer than M perhaps: all of them
            from = kLowest;
            if (!ok) {
                cut = find_cut_exact<TH>(n, s.M, most, key_of);
                by_place = cut.I < n;
            }
        }
    }
    floor = fmaxf(floor, ok ? from : key_value(cut.K).hi);
    for (int i = threadIdx.x; i < n; i += TH)
        if (ok ? s.score(i) >= from : kept(cut, key_of(i), i)) {
            const int k = atomicAdd(&c.count, 1);
            if (k < most) list[k] = i;
        }
    __syncthreads();
    return min(c.count, most);
}

// Sum of exp(c (z - m)) over a row by the whole block, for the beams whose order is in doubt. 2^t for t = c log2(e) (z - m) as a
// double-float: t = n + j / 256 + g with |g| <= 1 / 512, 2^(j / 256) from a table and 2^g - 1 (at most 0.0014) by three terms of
// its series in float32, 1.2e-10 off. Which thread adds which tokens in which order depends on their places in the row alone, so
// that rows with the same logits have the same sum however they lie in memory.
constexpr int kTable = 256;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: a sum with it is rounded to a whole number
__device__ __forceinline__ float2* exp_table(const BeamShared& s) { return s.at_offset<float2>(s.tail()); }
template <int TH>
__device__ __forceinline__ void fill_exp_table(const BeamParams& p, const BeamShared& s) {
    for (int j = threadIdx.x; j < kTable; j += TH) {
        const ddx e = exp_split(dd_mul_f(dd{SMCSD_LN2_HI, SMCSD_LN2_LO}, (float)j / 256.0f), p.T);
        const float u = pow2i(e.n);
        exp_table(s)[j] = make_float2(e.hi * u, e.lo * u);
    }
}
template <int DT, int TH>
__device__ __noinline__ dd precise_sum(const BeamParams& p, BeamShared s, BeamCounts& c, const void* row, float m) {
    constexpr int kEach = 8;
    const float2* table = exp_table(s);
    const dd c2 = dd_mul(dd{p.c_hi, p.c_lo}, dd{SMCSD_LOG2E_HI, SMCSD_LOG2E_LO});
    const int V = p.V;
    dd acc{0.0f, 0.0f};
    for (long long v0 = threadIdx.x; v0 < V; v0 += kEach * TH) {
        float z[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) z[k] = v0 + k * TH < V ? logit_at<DT>(row, v0 + k * TH) : kNegInf;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const dd d = two_sum(z[k], -m);
            const float th = fmaxf(f_mul(d.hi, c2.hi), -100.0f);  // what is smaller, a masked token among it, adds nothing, whatever the rest is
            const float tl = f_add(f_add(f_fma(d.hi, c2.hi, -th), f_mul(d.hi, c2.lo)), f_mul(d.lo, c2.hi));
            const float r = f_fma(th, 256.0f, kRound);  // 256 n + j in its last bits
            const int i = __float_as_int(r) - __float_as_int(kRound);
            const float g = f_add(f_fma(f_sub(r, kRound), -0.00390625f, th), th > -100.0f ? tl : 0.0f);
            const float e = f_mul(g, f_fma(g, f_fma(g, 0.0555041087f, 0.240226507f), 0.693147181f));
            const float2 t = table[i & 255];
            const float u = th > -100.0f ? __int_as_float(((i >> 8) + 127) << 23) : 0.0f;
            const dd a = two_sum(acc.hi, f_mul(t.x, u));
            acc.hi = a.hi;
            acc.lo = f_add(acc.lo, f_add(a.lo, f_mul(f_fma(t.x, e, t.y), u)));
        }
    }
    acc = warp_sum_dd(fast_two_sum(acc.hi, acc.lo));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) c.part[threadIdx.x >> 5] = acc;
    __syncthreads();
    acc = c.part[0];
    for (int w = 1; w < TH / 32; ++w) acc = dd_add(acc, c.part[w]);
    __syncthreads();
    return acc;
}

// log of a positive double-float: one step of Newton's method from the float logarithm, in double-floats.
__device__ __forceinline__ dd dd_log(dd v, const Exp2Table& T) {
    const float y = logf(v.hi);
    const ddx e = exp_split(dd{-y, 0.0f}, T);
    const float u = pow2i(e.n);  // v is at most 2^31
    const dd r = dd_add(dd_mul(v, dd{e.hi * u, e.lo * u}), dd{-1.0f, 0.0f});
    return dd_add(dd{y, 0.0f}, dd_add(r, dd{-0.5f * r.hi * r.hi, 0.0f}));
}

// log of a float to 4e-8: the exponent's part in double-floats, the mantissa's (of 0.75 to 1.5) by the float logarithm.
__device__ __forceinline__ dd dd_log_fast(float v) {
    const int k = (__float_as_int(v) - 0x3f400000) >> 23;
    const float m = __int_as_float(__float_as_int(v) - (k << 23));
    return dd_add(dd_mul_f(dd{SMCSD_LN2_HI, SMCSD_LN2_LO}, (float)k), dd{logf(m), 0.0f});
}

// Candidates by beam and token; kEnded stands for the token of a finished beam.
constexpr int kEnded = -1;
__device__ __forceinline__ uint64_t place_of(int beam, int token) { return (uint64_t)(uint32_t)beam << 32 | (uint32_t)token; }
__device__ __forceinline__ float start_score(const BeamParams& p, int g, int beam) {
    return p.scores ? __ldg(after_wait(p.scores) + (long long)g * p.N + beam) : 0.0f;
}

// Calls f(logit, beam, token) for every token of the sets in list2 whose logit is not below its beam's zmin. Half a warp takes a set,
// and four of them at a time, so that their loads are on the way together.
template <int DT, int TH, typename F>
__device__ __forceinline__ void scan_sets(const BeamParams& p, const BeamShared& s, int g, int n2, F&& f) {
    constexpr int PV = Geo<DT>::kPerVec, kEach = 4, kHalves = TH / 16;
    const int lane = threadIdx.x & 15, per = p.cpr * kBeamSets;
    for (int i0 = threadIdx.x >> 4; i0 < n2; i0 += kEach * kHalves) {
        uint4 x[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kHalves;
            if (i >= n2) break;
            const int set = s.list2()[i], l = (int)fast_div((uint32_t)set / kBeamSets, p.div_cpr);
            x[k] = beam_vec<DT>(beam_row<DT>(p, (long long)g * p.N + s.live(l)), (set - l * per) * 16 + lane);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kHalves;
            if (i >= n2) break;
            const int set = s.list2()[i], l = (int)fast_div((uint32_t)set / kBeamSets, p.div_cpr), beam = s.live(l);
            const float zmin = s.zmin(beam);
            float z[PV];
            unpack<DT>(x[k], z);
            unsigned hits = 0;
#pragma unroll
            for (int e = 0; e < PV; ++e) hits |= z[e] >= zmin ? 1u << e : 0u;
            if (hits) {
                const int v = (set - l * per) * 16 + lane, shift = beam_row<DT>(p, (long long)g * p.N + beam).shift;
                do {
                    const int e = __ffs(hits) - 1, w = DT == 0 ? e : e >> 1;
                    hits &= hits - 1;
                    const uint32_t word = w & 2 ? (w & 1 ? x[k].w : x[k].z) : (w & 1 ? x[k].y : x[k].x);
                    f(bits_to_float<DT>(DT == 0 ? word : (word >> (16 * (e & 1))) & 0xffffu), beam, (int)((long long)v * PV + e - shift));
                } while (hits);
            }
        }
    }
}

// Adds up one count a thread.
__device__ __forceinline__ unsigned long long block_total(BeamCounts& c, unsigned mine) {
    __syncthreads();
    if (threadIdx.x == 0) c.reduce = 0;
    __syncthreads();
    const unsigned w = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0 && w) atomicAdd(&c.reduce, (unsigned long long)w);
    __syncthreads();
    return c.reduce;
}

// More candidates than can be ranked, as where many tokens lie next to one another in the order: K and I so that those with a key
// above K, or with K and a place up to I, are at least M and no more than s.cands.
template <int DT, int TH>
__device__ __noinline__ void narrow_tokens(const BeamParams& p, BeamShared s, BeamCounts& c, int g, int n2, uint64_t* K, uint64_t* I) {
    const unsigned room = s.cands, M = p.M;
    uint64_t lo = *K, hi = ~0ull;
    const auto total = [&](uint64_t k, uint64_t i) {
        unsigned mine = 0;
        scan_sets<DT, TH>(p, s, g, n2, [&](float z, int beam, int token) {
            const uint64_t key = score_key(p, z, s.zmax(beam), s.base(beam));
            mine += key > k || (key == k && place_of(beam, token) <= i);
        });
        return block_total(c, mine);
    };
    while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        const unsigned long long n = total(mid, ~0ull);
        if (n > room) {
            lo = mid;
        } else if (n < M) {
            hi = mid;
        } else {
            *K = mid;
            return;
        }
    }
    *K = lo;
    uint64_t a = 0, b = place_of(p.N, 0);
    while (b - a > 1) {
        const uint64_t mid = a + (b - a) / 2;
        const unsigned long long n = total(lo, mid);
        if (n < M) {
            a = mid;
        } else {
            b = mid;
            if (n <= room) break;
        }
    }
    *I = b;
}

// Fills s.key, s.at with the candidates that can be among the first M; returns how many, and in `floor` the score below which
// candidates were left out (kLowest: none were). In a first turn the first level's maxima have been fetched to its scores, and
// scores are float32; in a second one they are exact.
template <int DT, int TH>
__device__ __forceinline__ int collect(const BeamParams& p, const BeamShared& s, BeamCounts& c, int g, bool exact, float& floor) {
    const int nlive = c.nlive;
    floor = kLowest;
    int n2 = 0;
    bool second = false;
    for (int sorted = 0;;) {
        const Level v = level_of<TH>(p, s, g, nlive, second, n2);
        const bool there = !second && !exact;  // fetched already, each by the thread that takes it now
#pragma unroll 2
        for (int i = threadIdx.x; i < v.n; i += TH) s.score(i) = level_score(p, s, v, i, there ? s.score(i) : v.z(s, i), exact);
        const float floor1 = floor;
        bool by_place;
        const int got = choose<TH>(s, c, v.n, float_of_order(c.best), 1.0f, LevelKey{&p, s, v}, v.log ? s.list2() : s.list1(), floor, by_place);
        if (second && by_place && !sorted) {
            // sets are chosen by their places, which follow the chunks': once more with the chunks in order
            sort_list<TH>(s.list1(), n2);
            floor = floor1;
            sorted = 1;
            continue;
        }
        if (second) {  // places in list1 to sets of the group's live beams
            for (int i = threadIdx.x; i < got; i += TH) s.list2()[i] = s.list1()[s.list2()[i] / kBeamSets] * kBeamSets + s.list2()[i] % kBeamSets;
            if (threadIdx.x == 0) c.chunks = n2;
        }
        n2 = got;
        if (v.log) break;
        second = true;
    }
    // the floor as a logit of each live beam, lowered by more than its roundings
    for (int l = threadIdx.x; l < nlive; l += TH) {
        const int beam = s.live(l);
        const float b = s.base(beam).x, m = s.zmax(beam), z = m + (floor - b) / p.c_hi;
        s.zmin(beam) = floor > kLowest ? fmaxf(z - (fabsf(m) + (fabsf(floor) + fabsf(b)) / p.c_hi) * 1e-6f - 1e-35f, kLowest) : kLowest;
    }
    __syncthreads();
    if (threadIdx.x == 0) c.count = 0;
    __syncthreads();
    const int room = s.cands;
    scan_sets<DT, TH>(p, s, g, n2, [&](float z, int beam, int token) {
        const int k = atomicAdd(&c.count, 1);
        if (k < room) s.key(k) = __float_as_uint(z), s.at(k) = place_of(beam, token);
    });
    __syncthreads();
    if (threadIdx.x == 0) c.narrowed = c.count > room;
    if (c.count <= room) {
        for (int i = threadIdx.x; i < c.count; i += TH) {
            const int beam = (int)(s.at(i) >> 32);
            s.key(i) = score_key(p, __uint_as_float((uint32_t)s.key(i)), s.zmax(beam), s.base(beam));
        }
    } else {
        uint64_t K = 1, I = ~0ull;  // kept: keys above K, and those equal to K up to place I
        narrow_tokens<DT, TH>(p, s, c, g, n2, &K, &I);
        floor = key_value(K).hi;
        __syncthreads();
        if (threadIdx.x == 0) c.count = 0;
        __syncthreads();
        scan_sets<DT, TH>(p, s, g, n2, [&](float z, int beam, int token) {
            const uint64_t key = score_key(p, z, s.zmax(beam), s.base(beam));
            if (key > K || (key == K && place_of(beam, token) <= I)) {
                const int k = atomicAdd(&c.count, 1);
                if (k < room) s.key(k) = key, s.at(k) = place_of(beam, token);
            }
        });
        __syncthreads();
    }
    const int got = min(c.count, room);
    for (int i = threadIdx.x; i < c.nover; i += TH) {
        const int beam = s.over(i);
        s.key(got + i) = key_of(dd{s.base(beam).x, s.base(beam).y});
        s.at(got + i) = place_of(beam, kEnded);
    }
    __syncthreads();
    return got + c.nover;
}

// Marks the beams of ranges that may have been left out though they come next to the last of the M best, whose beam and score are
// given; whether there are any of other beams. (Ranges that were kept are looked at token by token.)
template <int TH>
__device__ __noinline__ bool mark_near(const BeamParams& p, BeamShared s, BeamCounts& c, int g, int of, float last) {
    bool found = false;
    const auto mark = [&](int beam, float x) {
        if (beam == of || !(fabsf(x - last) <= doubt_of(c, last))) return;
        s.unsure(beam) = s.unsure(of) = 1;
        found = true;
    };
    for (int second = 0; second < 2; ++second) {
        const Level v = level_of<TH>(p, s, g, c.nlive, second, c.chunks);
        for (int i = threadIdx.x; i < v.n; i += TH) mark(v.beam(s, i), level_score(p, s, v, i, v.z(s, i), false));
        if (v.log) break;
    }
    if (c.narrowed)
        for (int l = threadIdx.x; l < c.nlive; l += TH) mark(s.live(l), last);
    return found;
}

// Ranks the candidates: s.order holds the first M (and one more, if there is one). Whether scores of different beams that
// decide about this order are nearer than the sums are good for; s.unsure marks those beams.
template <int TH>
__device__ __forceinline__ bool rank_and_doubt(const BeamParams& p, const BeamShared& s, BeamCounts& c, int g, int n, float floor) {
    for (int i = threadIdx.x; i < n; i += TH) {
        const uint64_t key = s.key(i), at = s.at(i);
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += s.key(j) > key || (s.key(j) == key && s.at(j) < at);
        if (rank <= p.M) s.order(rank) = i;
    }
    __syncthreads();
    if (c.nlive + c.nover <= 1) return false;
    for (int i = threadIdx.x; i < p.N; i += TH) s.unsure(i) = 0;
    __syncthreads();
    bool doubt = false;
    const auto near = [&](int i, int j) {
        const uint64_t a = s.at(i), b = s.at(j);
        if (a >> 32 == b >> 32 || ((int)(uint32_t)a == kEnded && (int)(uint32_t)b == kEnded)) return false;  // of one beam; exact
        const dd d = dd_sub(key_value(s.key(i)), key_value(s.key(j)));
        if (!(fabsf(d.hi) <= kTol)) return false;
        s.unsure((int)(a >> 32)) = s.unsure((int)(b >> 32)) = 1;
        return true;
    };
    const int m = min(p.M, n);
    for (int r = threadIdx.x; r < m && r + 1 < n; r += TH) doubt |= near(s.order(r), s.order(r + 1));
    if (n > p.M) {  // what is next to the last one, on either side, in any beam
        const int last = s.order(p.M - 1);
        for (int i = threadIdx.x; i < n; i += TH) doubt |= near(i, last);
    }
    if (floor > kLowest && n >= p.M) {  // and what was left out
        const float last = key_value(s.key(s.order(p.M - 1))).hi;
        if (last - floor <= doubt_of(c, floor)) doubt |= mark_near<TH>(p, s, c, g, (int)(s.at(s.order(p.M - 1)) >> 32), last);
    }
    return __syncthreads_or(doubt);
}

struct Mass {
    float m, s;
};
// Maximum and sum of a row's chunks, by one warp; NaN and +inf show in the sum.
__device__ __forceinline__ Mass row_mass(const BeamParams& p, long long row) {
    const int lane = threadIdx.x & 31;
    const float* qm = ws_ptr<const float>(p.ws, p.maxima) + row * p.cpr;
    const float* qs = ws_ptr<const float>(p.ws, p.sums) + row * p.cpr;
    float m = kNegInf, sum = 0.0f, first[3][2];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const bool in = k * 32 + lane < p.cpr;
        first[k][0] = in ? __ldcg(qm + k * 32 + lane) : kNegInf;
        first[k][1] = in ? __ldcg(qs + k * 32 + lane) : 0.0f;
        m = fmaxf(m, first[k][0]);
    }
    for (int k = 96 + lane; k < p.cpr; k += 32) m = fmaxf(m, __ldcg(qm + k));
    m = warp_max(m);
    const auto part = [&](float km, float ks) { return km > kNegInf ? ks * exp2f((km - m) * p.c2) : ks; };  // of -inf: 0, or NaN
#pragma unroll
    for (int k = 0; k < 3; ++k) sum += part(first[k][0], first[k][1]);
    for (int k = 96 + lane; k < p.cpr; k += 32) sum += part(__ldcg(qm + k), __ldcg(qs + k));
    return Mass{m, warp_sum(sum)};
}

// A beam's constant from its sum, by whole warps: s_i - log S_i, or none if there is no mass.
__device__ __forceinline__ void set_base(const BeamParams& p, const BeamShared& s, BeamCounts& c, int g, int beam, float m, dd sum, bool exact) {
    dd base{kNegInf, 0.0f};
    if (sum.hi > 0.0f) base = dd_sub(dd{start_score(p, g, beam), 0.0f}, exact ? dd_log(sum, p.T) : dd_log_fast(sum.hi));
    if ((threadIdx.x & 31) == 0) {
        s.zmax(beam) = m;
        s.base(beam) = make_float2(base.hi, base.lo);
        if (sum.hi > 0.0f) atomicMax(&c.best, float_order(base.hi));
    }
}

// The group's selection, by the last block of the group.
template <int DT, int TH>
__device__ __forceinline__ void beam_finish(const BeamParams& p, const BeamShared& s, BeamCounts& c, int g) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long rows = (long long)g * p.N;
    {   // the first level's maxima, for which nothing has to be known yet
        const Level v = level_of<TH>(p, s, g, c.nlive, false, 0);
#pragma unroll 4
        for (int i = threadIdx.x; i < v.n; i += TH) s.score(i) = v.z(s, i);
    }
    // a warp a beam: maximum and sum of its chunks
    for (int l = warp; l < c.nlive; l += TH / 32) {
        const int beam = s.live(l);
        const Mass a = row_mass(p, rows + beam);
        const float m = a.m, sum = a.s;
        const bool good = sum < kPosInf && m < kPosInf;
        if (!good && lane == 0) raise_error(p.ws, kErrNonfinite);
        set_base(p, s, c, g, beam, m, dd{good ? sum : 0.0f, 0.0f}, false);
    }
    // the beams' constants: scores are c (z - m) + base
    for (int i = threadIdx.x; i < c.nover; i += TH) {
        const float score = start_score(p, g, s.over(i));
        s.base(s.over(i)) = make_float2(score, 0.0f);
        atomicMax(&c.best, float_order(score));
    }
    __syncthreads();
    bool precise = false;
    int n;
    for (;;) {
        float floor;
        n = collect<DT, TH>(p, s, c, g, precise, floor);
        const bool doubt = rank_and_doubt<TH>(p, s, c, g, n, floor);
        if (!doubt || precise) break;
        precise = true;
        fill_exp_table<TH>(p, s);
        __syncthreads();
        for (int l = 0; l < c.nlive; ++l) {
            const int beam = s.live(l);
            if (!s.unsure(beam) || !(s.base(beam).x > kNegInf)) continue;  // the same for all threads
            const dd sum = precise_sum<DT, TH>(p, s, c, beam_row<DT>(p, rows + beam).row, s.zmax(beam));
            __syncthreads();
            set_base(p, s, c, g, beam, s.zmax(beam), sum, true);
            __syncthreads();
        }
    }
    for (int r = threadIdx.x; r < p.M; r += TH) {
        int token = p.pad, beam = 0, over = 1;
        float score = kNegInf;
        if (r < n && s.key(s.order(r))) {
            const uint64_t at = s.at(s.order(r));
            beam = (int)(at >> 32);
            if ((int)(uint32_t)at == kEnded) {
                score = start_score(p, g, beam);
            } else {
                token = (int)(uint32_t)at;
                score = key_value(s.key(s.order(r))).hi;
                over = p.eos >= 0 && token == p.eos;
            }
        }
        const long long o = (long long)g * p.M + r;
        p.tokens[o] = token;
        p.ancestors[o] = beam;
        p.out_scores[o] = score;
        if (p.out_finished) p.out_finished[o] = over;
    }
}

// ------------------------------------------------------------------------------------------
// groups of one: a row's M best tokens go by their logits alone, and are known without the row's sum
// ------------------------------------------------------------------------------------------

__device__ __forceinline__ uint64_t token_key(float z, int token) { return (uint64_t)float_order(z + 0.0f) << 32 | (uint32_t)~token; }
// A place's key where only logits count.
struct RowKey {
    BeamShared s;
    __device__ __forceinline__ uint64_t operator()(int i) const {
        const float x = s.score(i);
        return x > kNegInf ? (uint64_t)float_order(x + 0.0f) << 32 : 0;
    }
};

// A key that M to s.cands of the tokens of the sets in list2 are not below.
template <int DT, int TH>
__device__ __noinline__ uint64_t narrow_row(const BeamParams& p, BeamShared s, BeamCounts& c, int g, int n2) {
    uint64_t lo = 0, hi = ~0ull;
    while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        unsigned mine = 0;
        scan_sets<DT, TH>(p, s, g, n2, [&](float z, int, int token) { mine += token_key(z, token) >= mid; });
        const unsigned long long n = block_total(c, mine);
        if (n > (unsigned)s.cands)
            lo = mid;
        else if (n < (unsigned)s.M)
            hi = mid;
        else
            return mid;
    }
    return hi;
}

template <int DT, int TH>
__device__ __forceinline__ void row_finish(const BeamParams& p, const BeamShared& s, BeamCounts& c, int g) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    if (c.nlive) {
        const bool direct = p.cpr <= beam_keys(s, p.cpr, TH) / kBeamSets;
        const int n0 = direct ? p.cpr * kBeamSets : p.cpr;
        const float* sets = ws_ptr<const float>(p.ws, p.sets) + (long long)g * p.cpr * kBeamSets;
        const float* maxima = direct ? sets : ws_ptr<const float>(p.ws, p.maxima) + (long long)g * p.cpr;
#pragma unroll 4
        for (int i = threadIdx.x; i < n0; i += TH) s.score(i) = __ldcg(maxima + i);
        if (warp == 0) {
            const Mass a = row_mass(p, g);
            const bool good = a.s < kPosInf && a.m < kPosInf;
            if (!good && lane == 0) raise_error(p.ws, kErrNonfinite);
            set_base(p, s, c, g, 0, a.m, dd{good ? a.s : 0.0f, 0.0f}, false);
        }
        __syncthreads();
        if (s.base(0).x > kNegInf) {
            const float best = s.zmax(0), unit = 1.0f / p.c_hi;
            float floor = kLowest;
            int n2 = 0;
            bool second = false;
            for (int sorted = 0;;) {
                const bool sets_now = direct || second;
                const int n1 = second ? n2 * kBeamSets : n0;
                if (second) {
#pragma unroll 2
                    for (int i = threadIdx.x; i < n1; i += TH) s.score(i) = __ldcg(sets + s.list1()[i / kBeamSets] * kBeamSets + i % kBeamSets);
                }
                const float floor1 = floor;
                bool by_place;
                const int got = choose<TH>(s, c, n1, best, unit, RowKey{s}, sets_now ? s.list2() : s.list1(), floor, by_place);
                if (second && by_place && !sorted) {
                    // sets are chosen by their places, which follow the chunks': once more with the chunks in order
                    sort_list<TH>(s.list1(), n2);
                    floor = floor1;
                    sorted = 1;
                    continue;
                }
                if (second)
                    for (int i = threadIdx.x; i < got; i += TH) s.list2()[i] = s.list1()[s.list2()[i] / kBeamSets] * kBeamSets + s.list2()[i] % kBeamSets;
                n2 = got;
                if (sets_now) break;
                second = true;
            }
            if (threadIdx.x == 0) s.zmin(0) = floor;
            uint64_t K = 0;
            for (int turn = 0; turn < 2; ++turn) {
                __syncthreads();
                if (threadIdx.x == 0) c.count = 0;
                __syncthreads();
                scan_sets<DT, TH>(p, s, g, n2, [&](float z, int, int token) {
                    const uint64_t key = token_key(z, token);
                    if (key >= K) {
                        const int k = atomicAdd(&c.count, 1);
                        if (k < s.cands) s.key(k) = key;
                    }
                });
                __syncthreads();
                if (c.count <= s.cands) break;
                K = narrow_row<DT, TH>(p, s, c, g, n2);
            }
            n = min(c.count, s.cands);
            for (int i = threadIdx.x; i < n; i += TH) {
                const uint64_t key = s.key(i);
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) rank += s.key(j) > key;
                if (rank < p.M) s.order(rank) = i;
            }
        }
        __syncthreads();
    }
    for (int r = threadIdx.x; r < p.M; r += TH) {
        int token = p.pad, over = 1;
        float score = kNegInf;
        if (r < n) {
            const uint64_t key = s.key(s.order(r)), x = score_key(p, float_of_order((uint32_t)(key >> 32)), s.zmax(0), s.base(0));
            if (x) {  // else its score lies below float32's range, and those of all tokens behind it
                token = (int)~(uint32_t)key;
                score = key_value(x).hi;
                over = p.eos >= 0 && token == p.eos;
            }
        } else if (r == 0 && c.nover) {
            score = start_score(p, g, 0);
        }
        const long long o = (long long)g * p.M + r;
        p.tokens[o] = token;
        p.ancestors[o] = 0;
        p.out_scores[o] = score;
        if (p.out_finished) p.out_finished[o] = over;
    }
}

template <int DT, int TH, bool ONE>
__global__ void __launch_bounds__(TH, TH == kBeamWide ? 1 : ONE ? 8 : 5) beam_kernel(const __grid_constant__ BeamParams p) {
    __shared__ BeamCounts c;
    griddep_wait();
    const BeamShared s = beam_shared(p.N, p.M);
    constexpr int kWarps = TH / 32;
    const int g = blockIdx.x / p.blocks, b = blockIdx.x - g * p.blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {  // beams in order: those whose rows are read, and the finished ones
        int live = 0, over = 0;
        for (int i0 = 0; i0 < p.N; i0 += 32) {
            const int i = i0 + lane;
            const float score = i < p.N ? start_score(p, g, i) : kNegInf;
            if (!(score < kPosInf) && b == 0) raise_error(p.ws, kErrNonfinite);
            const bool some = score > kNegInf && score < kPosInf;
            const bool ended = some && p.finished && __ldg(after_wait(p.finished) + (long long)g * p.N + i);
            const unsigned l = __ballot_sync(0xffffffffu, some && !ended), o = __ballot_sync(0xffffffffu, ended);
            const unsigned before = (1u << lane) - 1u;
            if (some && !ended) s.live(live + __popc(l & before)) = i;
            if (ended) s.over(over + __popc(o & before)) = i;
            live += __popc(l);
            over += __popc(o);
        }
        if (lane == 0) c.nlive = live, c.nover = over, c.best = 0;
    }
    __syncthreads();
    const int items = c.nlive * p.cpr;
    for (int i = b * kWarps + warp; i < items; i += p.blocks * kWarps) {
        const int l = i / p.cpr, chunk = i - l * p.cpr;
        const long long row = (long long)g * p.N + s.live(l), at = row * p.cpr + chunk;
        beam_chunk<DT>(p, beam_row<DT>(p, row), chunk, ws_ptr<float>(p.ws, p.maxima) + at, ws_ptr<float>(p.ws, p.sums) + at,
                       ws_ptr<float>(p.ws, p.sets) + at * kBeamSets, lane);
    }
    __syncthreads();
    if (p.blocks > 1) {
        if (threadIdx.x == 0) {
            unsigned* count = ws_ptr<unsigned>(p.ws, kFrontGroup) + g;
            c.last = atom_add_release(count, 1u) == (unsigned)p.blocks - 1u;
            if (c.last) {
                fence_acquire();
                atomicExch(count, 0u);
            }
        }
        __syncthreads();
        if (!c.last) return;
    }
    griddep_launch_dependents();  // not before: blocks that wait beside the reading cost more (8 x 16 beams, three calls: 28.4 us for 26.7)
    if constexpr (ONE)
        row_finish<DT, TH>(p, s, c, g);
    else
        beam_finish<DT, TH>(p, s, c, g);
}

template <int DT, int TH, bool ONE>
static cudaError_t launch_beam_as(const BeamParams& p, cudaStream_t st) {
    const size_t shared = beam_shared_bytes(p.N, p.M, p.N * p.cpr, TH);
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(beam_kernel<DT, TH, ONE>), shared);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
    }
    return launch_waiting(beam_kernel<DT, TH, ONE>, dim3((unsigned)p.G * (unsigned)p.blocks), TH, shared, 0, st, p);
}

cudaError_t launch_beam(const BeamParams& p0, int dtype, cudaStream_t st) {
    BeamParams p = p0;
    const int sms = device_sm_count();
    // Blocks of 512 threads / of 128, us for groups of one beam of 32000 bf16: 152 groups 8.0 / 12.9, 160 14.0 / 12.8, 304 14.8 / 13.2, 400 21.5 /
    // 13.5; of 128256: 152 14.2 / 30.9, 160 25.6 / 31.7, 304 28.0 / 38.1, 400 43.3 / 43.8, 457 53.9 / 45.2, 1000 99.5 / 58.8; of 8 beams of 32000:
    // 152 27 / 67, 304 54 / 78, 457 100 / 91. The larger blocks have one SM each: their time steps up at 77, 153, 305 and 457 groups.
    const bool many = p.G >= 2 * sms || p.G > kFrontSeqs;  // the front has counters for that many groups
    // few groups: a chunk for each warp, as long as all blocks run at the same time
    const long long chunks = (long long)p.N * p.cpr, want = (chunks + kBeamWide / 32 - 1) / (kBeamWide / 32);
    const long long fit = many ? 1 : (long long)sms / p.G;
    p.blocks = (int)(want < fit ? want : fit);
    if (p.blocks < 1) p.blocks = 1;
    const auto launch = many ? dtype == 0 ? p.N == 1 ? launch_beam_as<0, kBeamNarrow, true> : launch_beam_as<0, kBeamNarrow, false>
                                          : p.N == 1 ? launch_beam_as<1, kBeamNarrow, true> : launch_beam_as<1, kBeamNarrow, false>
                             : dtype == 0 ? p.N == 1 ? launch_beam_as<0, kBeamWide, true> : launch_beam_as<0, kBeamWide, false>
                                          : p.N == 1 ? launch_beam_as<1, kBeamWide, true> : launch_beam_as<1, kBeamWide, false>;
    return launch(p, st);
}

}  // namespace smcsd
