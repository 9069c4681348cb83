// Selection of the pages that a sequence's new token reads, by a bound on its scores.
//
// A page scores sum_i a_i kmax_i + b_i kmin_i with a_i, b_i the sums of the positive and negative query channels of the kv
// head's group: one dot product of 2d terms for the whole group, bound by the bytes of the bounds. Which page comes in
// is to follow the float64 score, so that no rounding decides it; formed in float64 for every page it would be bound by
// its instructions (3.5 a channel). So every page is scored in float32 with a bound on the error, and only pages that
// float32 cannot tell from the n-th largest are scored again in float64 (a page or two of thousands; where there are
// many, as among equal pages, all of them).
//
// Two kernels. The first scores: all pages of all (sequence, kv head) rows form one line, cut evenly over the warps of
// all SMs, because one SM draws at most ~45 GB/s from DRAM however much it has in flight (a cluster of blocks per row
// left most SMs idle in a ragged batch: 32 sequences of 100 .. 65536 keys took 50 .. 114 us). The second has a block per
// row: it counts the scores into 2048 bins over their own range to find the bin of the n-th largest, ranks that bin's
// few pages one by one and writes the pages in order.
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "sm100.cuh"

namespace splitkv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kLoads = 8;         // copies of 16 bytes of bounds a lane makes in a round
constexpr int kStages = 3;        // rounds in flight and in use
constexpr int kRing = kWarps * kStages * kLoads * 32;  // 16-byte pieces: 192 KB
// Scores that the second kernel keeps in shared memory (192 KB, or 92 where two blocks share an SM); longer rows stay in L2. 8
// rows of 18750 pages: 36 us so, from L2 50; 16 rows of 43750: 112, 146.
template <int kPerSm>
constexpr int kInShared = kPerSm == 1 ? 49152 : 23552;
constexpr int kCands = 512;       // pages that are ranked one by one
constexpr int kWords = 512, kSpan = kWords * 32;
static_assert(kWords == kThreads && kCands <= kThreads, "one word, one candidate a thread");

// The order of the scores as unsigned integers: larger score, larger key, all above 0. NaN: below every number.
__device__ __forceinline__ uint64_t score_key(double s) {
    if (s != s) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);  // -0 ranks as 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ uint32_t score_key(float s) {
    if (s != s) return 1;
    const uint32_t u = __float_as_uint(s + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t u) { return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ float max_nan(float x, float y) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// The channels in 16 bytes of bounds or queries, exact in float32.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4& x, float (&f)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    // The larger sizes, channel by channel, as the type's bits (infinities above all numbers, NaN above them).
    static __device__ __forceinline__ uint32_t larger(uint32_t size, uint32_t x) { return __vmaxu2(size, x & 0x7fff7fffu); }
};
template <>
struct Chunk<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4& x, float (&f)[4]) {
        f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y), f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t size, uint32_t x) { return max(size, x & 0x7fffffffu); }
};

// How many pages of a sequence have to be scored, and which are taken without: pages < lead and >= tail.
struct Row {
    int32_t count, want, lead, tail;
    bool scored;
};
__device__ __forceinline__ Row row_of(const PagedMeta& m, int32_t len, int32_t n_select, int32_t keep_first,
                                      int32_t keep_last) {
    Row r;
    r.count = (len + m.page - 1) >> m.page_shift;
    r.want = min(n_select, r.count);
    r.lead = min(keep_first, r.count);
    r.tail = max(r.count - keep_last, r.lead);
    r.scored = r.count > n_select && r.lead + r.count - r.tail < r.want;
    return r;
}

// ---- first kernel: {key of the float32 score (0: not ranked), bound on the sums of terms' sizes} of every page. The
// bound stands with the last page of a warp's share, for all of the share: the sum over the channels of the coefficient's
// size times the largest size among the pages (2 instructions a pair of channels; a sum per page would take 4).
// LP lanes hold the 2d channels of one page, NC chunks of 16 bytes each.
template <typename T, int LP, int NC>
__global__ void __launch_bounds__(kThreads) score_kernel(PagedMeta m, const T* q, int64_t q_stride, const T* bounds,
                                                         const int32_t* table, const int32_t* seq_len, int32_t n_select,
                                                         int32_t keep_first, int32_t keep_last, uint2* scores,
                                                         int32_t* status) {
    constexpr int kN = Chunk<T>::kN, kPer = 32 / LP;    // pages a warp reads with one load a lane
    constexpr int kV = kLoads / NC, kStep = kV * kPer;  // pages of a lane's round, of a warp's
    static_assert(kStep <= 32 && LP >= kV, "one table entry, one result a lane");
    extern __shared__ uint4 smem[];
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + kRing);  // pages to score of the sequences before b
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint4* const ring = smem + warp * (kStages * kLoads * 32) + lane;
    after_previous();
    const bool bad = status_bad(status);
    auto pages_of = [&](int b) {
        const Row r = row_of(m, paged_len(m, seq_len, b, status), n_select, keep_first, keep_last);
        return r.scored ? r.count : 0;
    };
    if (m.n_seqs <= 32) {  // each warp by itself
        int32_t x = lane < m.n_seqs ? pages_of(lane) : 0;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, s);
            if (lane >= s) x += y;
        }
        prefix += warp * 36;
        prefix[lane + 1] = x;
        if (lane == 0) prefix[0] = 0;
        __syncwarp();
    } else {
        for (int b = tid; b < m.n_seqs; b += kThreads) prefix[b + 1] = pages_of(b);
        __syncthreads();
        if (warp == 0) {
            int32_t carry = 0;
            for (int b0 = 0; b0 < m.n_seqs; b0 += 32) {
                int32_t x = b0 + lane < m.n_seqs ? prefix[b0 + lane + 1] : 0;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int32_t y = __shfl_up_sync(0xffffffffu, x, s);
                    if (lane >= s) x += y;
                }
                if (b0 + lane < m.n_seqs) prefix[b0 + lane + 1] = carry + x;
                carry += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) prefix[0] = 0;
        }
        __syncthreads();
    }
    if (__any_sync(0xffffffffu, bad)) return;
    const int64_t total = (int64_t)prefix[m.n_seqs] * m.hkv;
    const int32_t n_warps = gridDim.x * kWarps, me = warp * gridDim.x + blockIdx.x;  // neighbours on other SMs
    const int64_t per = max((total + n_warps - 1) / n_warps, (int64_t)kStep);
    const int64_t u_end = min((me + 1) * per, total);
    const int sub = lane % LP, at = lane / LP;  // the lane's part of a page, its page of the kPer
    const int64_t page_step = (int64_t)m.hkv * 2 * m.d;

    for (int64_t u = me * per; u < u_end;) {
        // The rest of this warp's share of one (sequence, kv head): pages [p, p_end).
        int32_t b = 0;
        for (int32_t hi = m.n_seqs; hi - b > 1;) {
            const int32_t mid = (b + hi) >> 1;
            if ((int64_t)prefix[mid] * m.hkv <= u) b = mid; else hi = mid;
        }
        const int32_t count = prefix[b + 1] - prefix[b];
        const int64_t rem = u - (int64_t)prefix[b] * m.hkv;
        const int32_t g = rem >> 32 ? (int32_t)(rem / count) : (int32_t)((uint32_t)rem / (uint32_t)count);
        int32_t p = (int32_t)(rem - (int64_t)g * count);
        const int32_t p_end = (int32_t)min((int64_t)count, p + (u_end - u));
        u += p_end - p;
        const int32_t* trow = table + b * m.table_stride;
        const T* head = bounds + (int64_t)g * 2 * m.d;
        uint2* out = scores + ((int64_t)b * m.hkv + g) * m.max_pages;

        // Page-table entry p + lane, -1 for pages that are not ranked: those that are kept are not read either, as what their
        // bounds hold would widen the others' error bound (one that is not finite: to all pages of the row).
        auto entry = [&](int32_t p) {
            if (lane >= kStep || p + lane >= p_end) return -1;
            const int32_t page = paged_page(m, trow, p + lane, status);
            return p + lane < keep_first || p + lane >= count - keep_last ? -1 : page;
        };
        // Asynchronous copies into a ring of rounds in shared memory: two rounds are on their way while one is summed. (Loads
        // into registers one round ahead left the warps waiting for most of the time: 12 bytes a clock and SM.) A lane
        // reads back what it copied itself, so nothing has to be synchronised.
        auto fetch = [&](int32_t mine, int stage) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int32_t page = __shfl_sync(0xffffffffu, mine, v * kPer + at);
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const int e = (k * LP + sub) * kN;
                    const bool in = page >= 0 && e < 2 * m.d;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     sm100::smem_u32(ring + (stage * kLoads + v * NC + k) * 32)),
                                 "l"(in ? head + page * page_step + e : head), "r"(in ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int32_t ids[kStages + 1];  // table entries of this round and the next ones
#pragma unroll
        for (int r = 0; r <= kStages; ++r) ids[r] = entry(p + r * kStep);
        float c[NC][kN] = {};
        for (int h0 = 0; h0 < m.group; h0 += 4)
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int e = (k * LP + sub) * kN, i = e < m.d ? e : e - m.d;  // kmin's channels first, then kmax's
                uint4 y[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    y[h] = ldg_stream_if(q + b * q_stride + (int64_t)(g * m.group + h0 + h) * m.d + i,
                                         e < 2 * m.d && h0 + h < m.group);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float f[kN];
                    Chunk<T>::unpack(y[h], f);
#pragma unroll
                    for (int j = 0; j < kN; ++j) c[k][j] += (e < m.d) != (f[j] > 0.f) ? f[j] : 0.f;  // (NaN: into one of them)
                }
            }
#pragma unroll
        for (int r = 0; r < kStages - 1; ++r) fetch(ids[r], r);
        uint4 sizes[NC] = {};
        for (int stage = 0;; stage = stage + 1 < kStages ? stage + 1 : 0) {
            const int32_t after = entry(p + (kStages + 1) * kStep);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            uint4 x[kV][NC];
#pragma unroll
            for (int v = 0; v < kV; ++v)
#pragma unroll
                for (int k = 0; k < NC; ++k) x[v][k] = ring[(stage * kLoads + v * NC + k) * 32];
            fetch(ids[kStages - 1], stage == 0 ? kStages - 1 : stage - 1);
            float s[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                uint64_t sum = 0;  // of the even and of the odd channels
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    float f[kN];
                    Chunk<T>::unpack(x[v][k], f);
#pragma unroll
                    for (int j = 0; j < kN; j += 2)
                        sum = sm100::f2_fma(sm100::f2_pack(f[j], f[j + 1]), sm100::f2_pack(c[k][j], c[k][j + 1]), sum);
                    sizes[k].x = Chunk<T>::larger(sizes[k].x, x[v][k].x);
                    sizes[k].y = Chunk<T>::larger(sizes[k].y, x[v][k].y);
                    sizes[k].z = Chunk<T>::larger(sizes[k].z, x[v][k].z);
                    sizes[k].w = Chunk<T>::larger(sizes[k].w, x[v][k].w);
                }
                float even, odd;
                sm100::f2_unpack(sum, even, odd);
                s[v] = even + odd;
            }
            // Sums over the LP lanes; halving the values at each step while there are several: lane `sub` ends up
            // with the sum of value (sub * values / LP), the lanes of a value side by side.
#pragma unroll
            for (int step = LP / 2, have = kV; step; step >>= 1) {
                if (have > 1) {
                    have >>= 1;
#pragma unroll
                    for (int i = 0; i < kV / 2; ++i)
                        if (i < have) {
                            const float give = sub & step ? s[i] : s[i + have], keep = sub & step ? s[i + have] : s[i];
                            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, step);
                        }
                } else {
                    s[0] += __shfl_xor_sync(0xffffffffu, s[0], step);
                }
            }
            const int v = sub / (LP / kV), at_p = p + v * kPer + at;
            const int32_t page = __shfl_sync(0xffffffffu, ids[0], (v * kPer + at) & 31);
            if (sub % (LP / kV) == 0 && at_p < p_end) out[at_p] = make_uint2(page < 0 ? 0 : score_key(s[0]), 0);
            if ((p += kStep) >= p_end) break;
#pragma unroll
            for (int r = 0; r < kStages; ++r) ids[r] = ids[r + 1];
            ids[kStages] = after;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // (what runs past the share copies nothing)
        float size = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float f[kN];
            Chunk<T>::unpack(sizes[k], f);
#pragma unroll
            for (int j = 0; j < kN; ++j) size = fmaf(f[j], fabsf(c[k][j]), size);
        }
#pragma unroll
        for (int step = LP / 2; step; step >>= 1) size += __shfl_xor_sync(0xffffffffu, size, step);
#pragma unroll
        for (int step = 16; step >= LP; step >>= 1) size = max_nan(size, __shfl_xor_sync(0xffffffffu, size, step));
        __syncwarp();  // after the key beside it
        if (lane == 0) out[p_end - 1].y = __float_as_uint(size);
    }
}

// ---- second kernel

struct Shared {
    uint32_t hist[kBins];
    uint64_t cand_key[kCands];
    int32_t cand_page[kCands];
    uint64_t red[2 * kWarps];
    int32_t ired[kWarps];
    int32_t found[6];
    uint32_t in_mask[kWords], eq_mask[kWords];
};

// Sum of x over the threads before this one, and over all of them. Two barriers.
__device__ __forceinline__ int2 sum_before(int32_t x, int32_t* warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t incl = x;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    const int32_t w = lane < kWarps ? warps[lane] : 0;
    const int32_t below = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0), all = __reduce_add_sync(0xffffffffu, w);
    __syncthreads();
    return make_int2(below + incl - x, all);
}

// The keys of a row, of one width or the other.
template <typename K>
struct Keys {
    K* at;
    int32_t n, step;  // elements from one page's key to the next's
    template <typename F>
    __device__ __forceinline__ void each(F&& fn) const {  // pages over the threads
#pragma unroll 4
        for (int32_t p = threadIdx.x; p < n; p += kThreads) fn(p, at[(int64_t)p * step]);
    }
};

// Narrows [lo, hi], which holds all keys of interest, to a bin with the `need`-th largest of them; `need` then counts
// from the bin's top. Ends with at most kCands keys in the bin, or with all of them needed, or all equal. hist is zero
// before and after.
template <typename K>
__device__ __forceinline__ void narrow(const Keys<K>& keys, Shared& sh, K& lo, K& hi, int32_t& need, int32_t& in_bin) {
    const int tid = threadIdx.x;
    const K range = hi - lo;
    int shift = 0;
    if (lo < hi && range >> kBits)
        shift = 8 * (int)sizeof(K) - kBits - (sizeof(K) == 8 ? __clzll((long long)range) : __clz((int)range));
    for (;;) {
        if (tid < 4) sh.found[tid] = 0;
        __syncthreads();
        keys.each([&](int32_t, K k) {
            if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        });
        __syncthreads();
        // Thread t has the bins 4t .. 4t + 3 counted from the top.
        constexpr int kEach = kBins / kThreads;
        static_assert(kEach == 4, "one 16-byte load");
        uint4* bins = reinterpret_cast<uint4*>(sh.hist + kBins - kEach * (tid + 1));
        const uint4 y = *bins;
        *bins = make_uint4(0, 0, 0, 0);
        const uint32_t v[kEach] = {y.w, y.z, y.y, y.x};
        const int32_t sum = v[0] + v[1] + v[2] + v[3];
        int32_t above = sum_before(sum, sh.ired).x;
        if (above < need && above + sum >= need) {
            int k = 0;
#pragma unroll
            for (int i = 0; i < kEach - 1; ++i)
                if (k == i && above + (int32_t)v[i] < need) above += v[i], ++k;
            sh.found[0] = kBins - 1 - kEach * tid - k;
            sh.found[1] = above;
            sh.found[2] = k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3];
        }
        __syncthreads();
        need -= sh.found[1];
        in_bin = sh.found[2];
        lo += (K)sh.found[0] << shift;
        const K width = ((K)1 << shift) - 1;
        if (hi - lo > width) hi = lo + width;  // (the last bin may reach past the range)
        if (in_bin <= kCands || in_bin <= need || shift == 0) return;
        shift = max(0, shift - kBits);
        __syncthreads();
    }
}

// The keys in [from, to] into the list of candidates. Their number (those past kCands are only counted), and how many of
// them are above `mark`.
template <typename K>
__device__ __forceinline__ int2 gather(const Keys<K>& keys, Shared& sh, K from, K to, K mark) {
    if (threadIdx.x < 2) sh.found[4 + threadIdx.x] = 0;
    __syncthreads();
    keys.each([&](int32_t p, K k) {
        if (k >= from && k <= to) {
            const int32_t i = atomicAdd(&sh.found[4], 1);
            if (k > mark) atomicAdd(&sh.found[5], 1);
            if (i < kCands) sh.cand_key[i] = k, sh.cand_page[i] = p;
        }
    });
    __syncthreads();
    return make_int2(sh.found[4], sh.found[5]);
}

// How many of the n candidates come before this thread's: larger keys, equal keys of lower pages.
__device__ __forceinline__ int32_t place(const Shared& sh, int32_t n) {
    const uint64_t k = sh.cand_key[threadIdx.x];
    const int32_t p = sh.cand_page[threadIdx.x];
    int32_t better = 0;
    for (int j = 0; j < n; ++j) better += sh.cand_key[j] > k || (sh.cand_key[j] == k && sh.cand_page[j] < p);
    return better;
}

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(x.x << 16), f[1] = __uint_as_float(x.x & 0xffff0000u);
    f[2] = __uint_as_float(x.y << 16), f[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
}

// The key of page p's float64 score, on one warp: the group's query channels again, in float64.
template <typename T>
__device__ __forceinline__ uint64_t exact(const PagedMeta& m, const T* q, const T* head, const int32_t* trow, int32_t p,
                                       int32_t* status) {
    const int lane = threadIdx.x & 31;
    const int32_t page = paged_page(m, trow, p, status);
    if (page < 0) return 0;
    const T* x = head + page * ((int64_t)m.hkv * 2 * m.d);
    double s = 0.0;
    const int i = 4 * lane;  // d is a multiple of 4, at most 128: all loads at once
    if (i < m.d) {
        double up[4] = {}, down[4] = {};
        float lo[4], hi[4];
        load4(x + i, lo);
        load4(x + m.d + i, hi);
        for (int h0 = 0; h0 < m.group; h0 += 8) {
            float y[8][4];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                if (h0 + h < m.group) load4(q + (int64_t)(h0 + h) * m.d + i, y[h]);
                else y[h][0] = y[h][1] = y[h][2] = y[h][3] = 0.f;
            }
#pragma unroll
            for (int h = 0; h < 8; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    up[j] += y[h][j] > 0.f ? y[h][j] : 0.f;
                    down[j] += y[h][j] > 0.f ? 0.f : y[h][j];
                }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma((double)lo[j], down[j], s), s = fma((double)hi[j], up[j], s);
    }
#pragma unroll
    for (int y = 16; y; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
    return score_key(s);
}

// Writes the pages taken, in order: the kept ones, those with keys >= take, and of those in [lo, hi] the first `ties`.
template <typename K>
__device__ __forceinline__ void write_pages(const Keys<K>& keys, Shared& sh, const Row& r, K take, K lo, K hi,
                                         int32_t ties, int32_t* out, int32_t n_select) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t at_out = 0, left = ties;
    for (int32_t first = 0; first < r.count; first += kSpan) {
        const int32_t here = min(r.count - first, kSpan);
#pragma unroll 1
        for (int32_t i = warp * 32; i < here; i += kThreads) {
            const int32_t p = first + i + lane;
            const K key = p < r.count ? keys.at[(int64_t)p * keys.step] : 0;
            const bool kept = p < r.count && (p < r.lead || p >= r.tail);
            const uint32_t in = __ballot_sync(0xffffffffu, kept || (key && key >= take));
            if (ties) {
                const uint32_t eq = __ballot_sync(0xffffffffu, key >= lo && key <= hi);
                if (lane == 0) sh.eq_mask[i / 32] = eq;
            }
            if (lane == 0) sh.in_mask[i / 32] = in;
        }
        __syncthreads();
        uint32_t in = tid * 32 < here ? sh.in_mask[tid] : 0;
        if (ties) {  // of the equal ones the first
            uint32_t eq = tid * 32 < here ? sh.eq_mask[tid] : 0;
            const int2 before = sum_before(__popc(eq), sh.ired);
            for (int32_t i = before.x; eq && i < left; ++i) in |= eq & -eq, eq &= eq - 1;
            left -= min(left, before.y);
        }
        const int2 before = sum_before(__popc(in), sh.ired);
        int32_t pos = at_out + before.x;
        at_out += before.y;
        for (; in; in &= in - 1, ++pos)
            if (pos < n_select) out[pos] = first + tid * 32 + __ffs(in) - 1;
    }
    // Fewer than wanted only where pages out of range were not ranked.
    for (int32_t i = at_out + tid; i < n_select; i += kThreads) out[i] = -1;
}

// More pages than are ranked one by one cannot be told from the n-th largest: the scores of all of them in float64, in the
// place of the float32 ones, and those that are sure to be taken ~0. For equal pages (a query of zeros makes all equal) and
// scores that are not finite, on the row's one block: bound by the loads of table and bounds that each warp waits for, page
// after page. 8 rows of 4096 pages, d 128: 485 us where all are equal, 19 where they are not; of 400: 99 and 10; of 49152:
// 7.5 ms and 89 us.
template <typename T>
__device__ __noinline__ void pick_wide(const PagedMeta& m, const T* q, const T* head, const int32_t* trow, uint2* scores,
                                       Shared& sh, const Row& r, uint32_t from, uint32_t to, int32_t need, int32_t* out,
                                       int32_t n_select, int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Keys<uint64_t> wide{reinterpret_cast<uint64_t*>(scores), r.count, 1};
    uint64_t lo = ~0ull, hi = 0;
    for (int32_t p = warp; p < r.count; p += kWarps) {
        const uint32_t k = scores[p].x;
        const uint64_t x = k > to ? ~0ull : k >= from ? exact<T>(m, q, head, trow, p, status) : 0;
        __syncwarp();
        if (lane == 0) wide.at[p] = x;
        if (x && ~x) lo = min(lo, x), hi = max(hi, x);
    }
    if (lane == 0) sh.red[warp] = lo, sh.red[kWarps + warp] = hi;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) lo = min(lo, sh.red[w]), hi = max(hi, sh.red[kWarps + w]);
    int32_t in_bin;
    narrow(wide, sh, lo, hi, need, in_bin);
    int32_t ties = 0;
    uint64_t take = lo;
    if (in_bin > need) {
        take = hi + 1;
        if (in_bin <= kCands) {
            gather(wide, sh, lo, hi, hi);
            if (threadIdx.x < in_bin) wide.at[sh.cand_page[threadIdx.x]] = place(sh, in_bin) < need ? ~0ull : 0;
        } else {
            ties = need;
        }
        __syncthreads();
    }
    write_pages(wide, sh, r, take, lo, hi, ties, out, n_select);
}

// A float32 score's error over the sum of its terms' sizes: the coefficients' sums (G - 1), at most 8 terms in a lane's sum,
// 1 sum of two and 5 of lanes (14), each rounding 2^-24 of something no larger; the sizes' own sums as much.
__device__ __forceinline__ float error_of(const PagedMeta& m) { return (32 + 2 * m.group) * 0x1p-24f; }

// One block per (sequence, kv head). It runs once through code that nothing has run before, so what counts is how many
// instructions it has to fetch: loops stay loops. One block an SM (kPerSm = 1) has the registers that it needs (124, no
// spills; 104 bytes of stack, pick_wide's call among them); two have 64, with 24 to 40 bytes of spills. More rows than SMs
// want two there. 8 rows of 4096 pages, select as a whole: 14.2 us, 16.2 with two; 2048 rows of 250:
// 115 us, 94 with two.
template <typename T, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) pick_kernel(PagedMeta m, const T* q, int64_t q_stride,
                                                                const T* bounds, const int32_t* table,
                                                                const int32_t* seq_len, int32_t n_select,
                                                                int32_t keep_first, int32_t keep_last, uint2* scores,
                                                                int32_t* pages, int32_t* status) {
    extern __shared__ uint32_t copy[];
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x, b = row / m.hkv, g = row % m.hkv;
    scores += (int64_t)row * m.max_pages;
    after_previous();
    const Row r = row_of(m, paged_len(m, seq_len, b, status), n_select, keep_first, keep_last);
    constexpr int kAhead = kPerSm == 1 ? 8 : 4;  // scores of a thread that are loaded at once
    uint2 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = r.scored && i * kThreads + tid < r.count ? scores[i * kThreads + tid] : make_uint2(0, 0);
    const bool bad = status_bad(status);
    const int32_t* trow = table + b * m.table_stride;
    int32_t* out = pages + (int64_t)row * n_select;
    reinterpret_cast<uint4*>(sh.hist)[tid] = make_uint4(0, 0, 0, 0);
    if (__syncthreads_or(bad)) return;
    if (!r.scored) {
        for (int i = tid; i < n_select; i += kThreads)
            out[i] = i >= r.want ? -1 : r.count <= n_select || i < r.lead ? i : r.tail + i - r.lead;
        for (int i = tid; i < r.count; i += kThreads) paged_page(m, trow, i, status);  // checked all the same
        return;
    }
    Keys<uint32_t> keys{copy, r.count, 1};
    if (r.count > kInShared<kPerSm>) keys = {reinterpret_cast<uint32_t*>(scores), r.count, 2};
    uint32_t lo = ~0u, hi = 0;
    float size = 0.f;
    auto see = [&](int32_t p, const uint2& x) {
        if (keys.step == 1) copy[p] = x.x;
        lo = min(lo, x.x - 1), hi = max(hi, x.x);  // (0, not ranked, is the largest there)
        size = max_nan(size, __uint_as_float(x.y));
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i * kThreads + tid < r.count) see(i * kThreads + tid, x[i]);
    for (int32_t p = kAhead * kThreads + tid; p < r.count; p += kThreads) see(p, scores[p]);
    // Sizes are not negative: as integers they have the floats' order, NaN on top.
    static_assert(kWarps == 16, "two values a lane");
    lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(size) & 0x7fffffffu);
    if (lane == 0) sh.red[warp] = (uint64_t)hi << 32 | lo, sh.ired[warp] = (int32_t)most;
    __syncthreads();
    const uint64_t both = sh.red[lane % kWarps];
    lo = __reduce_min_sync(0xffffffffu, (uint32_t)both) + 1, hi = __reduce_max_sync(0xffffffffu, (uint32_t)(both >> 32));
    size = __uint_as_float(__reduce_max_sync(0xffffffffu, (uint32_t)sh.ired[lane % kWarps]));
    const float err = fmaf(size, 2.f * error_of(m), 0x1p-140f);  // twice the error (and what denormal terms may lose)
    if (lo == 0) lo = ~0u, hi = 0;                               // nothing ranked

    // The bin with the n-th largest; pages from 2 errors below it to 2 above cannot be told from the n-th largest.
    const int32_t open = r.want - (r.lead + r.count - r.tail);
    int32_t need = open, in_bin;
    narrow(keys, sh, lo, hi, need, in_bin);
    uint32_t from = 1, to = ~0u;
    const bool finite = in_bin && err < INFINITY;
    if (finite) {
        from = max(score_key(__fsub_rd(key_score(lo), err)), 1u);
        to = score_key(__fadd_ru(key_score(hi), err));
    }
    const int2 near = gather(keys, sh, from, to, hi);
    // Above them: what narrow() counted above the bin, without those that are near.
    need = finite ? need + near.y : in_bin ? open : near.x;
    uint32_t take = from;
    if (near.x > need) {
        const T* qg = q + b * q_stride + (int64_t)g * m.group * m.d;
        const T* head = bounds + (int64_t)g * 2 * m.d;
        if (near.x > kCands || !finite) {
            pick_wide<T>(m, qg, head, trow, scores, sh, r, from, to, need, out, n_select, status);
            return;
        }
        // The n-th largest itself; usually no other page is within 2 errors of it.
        const uint32_t mine = tid < near.x ? (uint32_t)sh.cand_key[tid] : 0;
        const int32_t before = tid < near.x ? place(sh, near.x) : INT32_MAX;
        if (before == need - 1) sh.found[0] = (int32_t)mine;
        __syncthreads();
        const float nth = key_score((uint32_t)sh.found[0]);
        const uint32_t below = score_key(__fsub_rd(nth, err)), above = score_key(__fadd_ru(nth, err));
        const int32_t sure = __syncthreads_count(mine > above), open2 = __syncthreads_count(mine && mine >= below) - sure;
        bool in = mine && mine >= below;
        if (sure + open2 > need) {  // the others in float64; those above come first, those below last
            for (int i = warp; i < near.x; i += kWarps) {
                const uint32_t k = (uint32_t)sh.cand_key[i];
                const uint64_t e = k > above ? ~0ull : k < below ? 0 : exact<T>(m, qg, head, trow, sh.cand_page[i], status);
                __syncwarp();
                if (lane == 0) sh.cand_key[i] = e;
            }
            __syncthreads();
            in = tid < near.x && place(sh, near.x) < need;
        }
        if (tid < near.x) keys.at[(int64_t)sh.cand_page[tid] * keys.step] = in ? ~0u : 0;
        take = to + 1;
        __syncthreads();
    }
    write_pages(keys, sh, r, take, 1u, 0u, 0, out, n_select);
}

template <typename T, int LP, int NC>
cudaError_t launch(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds, const int32_t* table,
                   const int32_t* seq_len, int32_t n_select, int32_t keep_first, int32_t keep_last, int32_t* pages,
                   int32_t* status, void* ws, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const bool many = (int64_t)m.n_seqs * m.hkv > sms;
    auto pick = many ? pick_kernel<T, 2> : pick_kernel<T, 1>;
    static SmemGrants granted[2];
    const int in_shared = many ? kInShared<2> : kInShared<1>;
    e = allow_smem((const void*)pick, sizeof(uint32_t) * in_shared, granted[many]);
    if (e != cudaSuccess) return e;
    auto score = score_kernel<T, LP, NC>;
    static SmemGrants score_granted;
    e = allow_smem((const void*)score, sizeof(uint4) * kRing + sizeof(int32_t) * (SPLITKV_PAGED_MAX_SEQS + 1), score_granted);
    if (e != cudaSuccess) return e;
    const size_t lens = sizeof(uint4) * kRing + sizeof(int32_t) * std::max(m.n_seqs + 1, kWarps * 36);
    e = launch_overlapped(score, sms, kThreads, lens, st, m, (const T*)q, q_stride, (const T*)k_bounds,
                          table, seq_len, n_select, keep_first, keep_last, (uint2*)ws, status);
    if (e == cudaSuccess)
        e = launch_overlapped(pick, m.n_seqs * m.hkv, kThreads, sizeof(uint32_t) * std::min(m.max_pages, in_shared), st, m,
                              (const T*)q, q_stride, (const T*)k_bounds, table, seq_len, n_select, keep_first,
                              keep_last, (uint2*)ws, pages, status);
    return note_error(e, "paged select");
}

}  // namespace

size_t paged_select_workspace(const PagedMeta& m) { return sizeof(uint2) * m.n_seqs * m.hkv * m.max_pages; }

cudaError_t launch_paged_select(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds,
                                const int32_t* table, const int32_t* seq_len, int32_t n_select, int32_t keep_first,
                                int32_t keep_last, int32_t* pages, int32_t* status, void* ws, cudaStream_t st) {
#define SPLITKV_SELECT(T, LP, NC) \
    launch<T, LP, NC>(m, q, q_stride, k_bounds, table, seq_len, n_select, keep_first, keep_last, pages, status, ws, st)
    const int chunks = 2 * m.d * (m.dtype == SPLITKV_BF16 ? 2 : 4) / 16;  // 16-byte pieces of a page's bounds
    if (m.dtype == SPLITKV_BF16) {
        if (chunks <= 8) return SPLITKV_SELECT(__nv_bfloat16, 8, 1);
        return chunks <= 16 ? SPLITKV_SELECT(__nv_bfloat16, 16, 1) : SPLITKV_SELECT(__nv_bfloat16, 32, 1);
    }
    if (chunks <= 8) return SPLITKV_SELECT(float, 8, 1);
    if (chunks <= 16) return SPLITKV_SELECT(float, 16, 1);
    return chunks <= 32 ? SPLITKV_SELECT(float, 32, 1) : SPLITKV_SELECT(float, 32, 2);
#undef SPLITKV_SELECT
}

}  // namespace splitkv
