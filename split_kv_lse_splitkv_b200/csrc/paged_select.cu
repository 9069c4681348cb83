// Selection of the pages that a sequence's new token reads, by a bound on its scores.
//
// A page scores sum_i a_i kmax_i + b_i kmin_i with a_i, b_i the sums of the positive and negative query channels of the kv
// head's group: one dot product of 2d terms for the whole group, bound by the bytes of the bounds. It is formed in
// float64 (bf16 or float32 channels enter exactly, the order of the sum moves it by 1e-16), so that which page comes
// in does not hang on a rounding. A cluster of blocks shares a (sequence, kv head): each block scores a run of pages
// and keeps their scores in shared memory as ordered integers; the n-th largest is found by counting into 2048 bins
// over the range that is left (the first pass spans the scores' own range, so two passes nearly always decide), the
// blocks adding up each other's bins through distributed shared memory; then each writes its pages in order.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace splitkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 8;        // loads of bounds a lane has in flight
constexpr int kMaxShare = 16384;  // pages of one block: 128 KB of scores
static_assert(kMaxShare * kMaxCluster >= kMaxSelectPages, "the longest sequence fits a cluster");

// The order of the scores as unsigned integers: larger score, larger key, all above 0. NaN: below every number.
__device__ __forceinline__ uint64_t score_key(double s) {
    if (s != s) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);  // -0 ranks as 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

template <typename T>
struct Chunk;  // 16 bytes of bounds
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ double dot(const uint4& x, const double (&c)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fma((double)__uint_as_float(w[i] << 16), c[2 * i], s);
            s = fma((double)__uint_as_float(w[i] & 0xffff0000u), c[2 * i + 1], s);
        }
        return s;
    }
};
template <>
struct Chunk<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ double dot(const uint4& x, const double (&c)[4]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma((double)__uint_as_float(w[i]), c[i], s);
        return s;
    }
};

// What the blocks of a cluster read of each other.
struct Shared {
    uint32_t hist[kBins];
    uint64_t least, most;   // keys of this block
    int32_t skip, above, equal;
};

// LP lanes hold the 2d channels of one page, NC chunks of 16 bytes each.
template <typename T, int LP, int NC>
__global__ void __launch_bounds__(kThreads) select_kernel(PagedMeta m, const T* __restrict__ q, int64_t q_stride,
                                                          const T* __restrict__ bounds,
                                                          const int32_t* __restrict__ table,
                                                          const int32_t* __restrict__ seq_len, int32_t n_select,
                                                          int32_t keep_first, int32_t keep_last,
                                                          int32_t* __restrict__ pages, int32_t* status, int32_t cl) {
    constexpr int kN = Chunk<T>::kN, kPer = 32 / LP;  // pages a warp reads with one load a lane
    extern __shared__ uint64_t keys[];                // of this block's pages; 0: not ranked
    __shared__ Shared sh;
    __shared__ double coef[256];
    __shared__ uint64_t red[2 * kWarps];
    __shared__ int32_t ired[2 * kWarps];
    __shared__ int32_t found[3];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % cl, row = blockIdx.x / cl, b = row / m.hkv, g = row % m.hkv;

    if (tid == 0) sh.skip = status_bad(status);
    const int32_t len = paged_len(m, seq_len, b, status);
    const int32_t count = (len + m.page - 1) >> m.page_shift, want = min(n_select, count);
    const int32_t lead = min(keep_first, count), tail = max(count - keep_last, lead);  // always taken: < lead, >= tail
    int32_t* out = pages + (int64_t)row * n_select;
    if (count <= n_select || lead + count - tail >= want) {  // no score decides (the same for the whole cluster)
        for (int i = rank * kThreads + tid; i < n_select; i += cl * kThreads)
            out[i] = i >= want ? -1 : count <= n_select || i < lead ? i : tail + i - lead;
        for (int i = rank * kThreads + tid; i < count; i += cl * kThreads)  // the pages are checked all the same
            paged_page(m, table + b * m.table_stride, i, status);
        return;
    }

    // ---- scores of pages [p0, p1)
    for (int i = tid; i < m.d; i += kThreads) {
        double up = 0.0, down = 0.0;
        const T* x = q + b * q_stride + (int64_t)g * m.group * m.d + i;
        for (int h = 0; h < m.group; ++h) {
            const double y = to_f32<T>(x[(int64_t)h * m.d]);
            up += y > 0.0 ? y : 0.0;
            down += y < 0.0 ? y : 0.0;
            if (y != y) up = down = y;
        }
        coef[i] = down;
        coef[m.d + i] = up;
    }
    const int32_t share = (count + cl - 1) / cl, p0 = min(rank * share, count), n = min(share, count - p0);
    const int32_t* trow = table + b * m.table_stride + p0;
    __syncthreads();
    const int sub = lane % LP, at = lane / LP;  // the lane's part of a page, its page of the kPer
    double c[NC][kN];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = (k * LP + sub) * kN + i;
            c[k][i] = e < 2 * m.d ? coef[e] : 0.0;
        }
    uint64_t least = ~0ull, most = 0;
    constexpr int kStep = kUnroll / NC * kPer;  // pages of a warp's round: kStep <= 32
    static_assert(kStep <= 32, "one table entry a lane");
    for (int32_t base = warp * kStep; base < n; base += kWarps * kStep) {
        const int32_t mine = lane < kStep && base + lane < n ? paged_page(m, trow, base + lane, status) : -1;
        uint4 x[kUnroll / NC][NC];
#pragma unroll
        for (int u = 0; u < kUnroll / NC; ++u) {
            const int32_t page = __shfl_sync(0xffffffffu, mine, u * kPer + at);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int e = (k * LP + sub) * kN;
                x[u][k] = page >= 0 && e < 2 * m.d
                              ? __ldg(reinterpret_cast<const uint4*>(bounds + ((int64_t)page * m.hkv + g) * 2 * m.d + e))
                              : make_uint4(0, 0, 0, 0);
            }
        }
        double s[kUnroll / NC];
#pragma unroll
        for (int u = 0; u < kUnroll / NC; ++u) {
            s[u] = 0.0;
#pragma unroll
            for (int k = 0; k < NC; ++k) s[u] += Chunk<T>::dot(x[u][k], c[k]);
        }
        // Sums over the LP lanes; halving the values at each step while there are several: lane `sub` ends up
        // with the sum of value (sub * values / LP), the lanes of a value side by side.
        constexpr int kV = kUnroll / NC;
#pragma unroll
        for (int step = LP / 2, have = kV; step; step >>= 1) {
            if (have > 1) {
                have >>= 1;
#pragma unroll
                for (int i = 0; i < kV / 2; ++i)
                    if (i < have) {
                        const double give = sub & step ? s[i] : s[i + have], keep = sub & step ? s[i + have] : s[i];
                        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, step);
                    }
            } else {
                s[0] += __shfl_xor_sync(0xffffffffu, s[0], step);
            }
        }
        static_assert(LP >= kV, "every value of a round gets a lane");
        const int u = sub / (LP / kV);
        const int32_t p = base + u * kPer + at;
        const int32_t page = __shfl_sync(0xffffffffu, mine, (u * kPer + at) & 31);
        if (sub % (LP / kV) == 0 && p < n) {
            const bool kept = p0 + p < lead || p0 + p >= tail;
            const uint64_t key = kept || page < 0 ? 0 : score_key(s[0]);
            keys[p] = key;
            if (key) least = min(least, key), most = max(most, key);
        }
    }

    // ---- the scores' range
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        least = min(least, __shfl_xor_sync(0xffffffffu, least, x));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
    }
    if (lane == 0) red[warp] = least, red[kWarps + warp] = most;
    __syncthreads();
    if (warp == 0) {
        least = lane < kWarps ? red[lane] : ~0ull;
        most = lane < kWarps ? red[kWarps + lane] : 0;
#pragma unroll
        for (int x = 8; x; x >>= 1) {
            least = min(least, __shfl_xor_sync(0xffffffffu, least, x));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
        }
        if (lane == 0) sh.least = least, sh.most = most;
    }
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    cluster.sync();
    const int skip = cluster.map_shared_rank(&sh, 0)->skip;  // one block's word decides for all of them
    uint64_t lo = ~0ull, hi = 0;
    for (int r = 0; r < cl; ++r) {
        const Shared* x = cluster.map_shared_rank(&sh, r);
        lo = min(lo, x->least);
        hi = max(hi, x->most);
    }
    if (skip || lo > hi) {  // nothing ranked: every page in use is out of range
        cluster.sync();
        return;
    }

    // ---- the `need` largest keys: [lo, hi] is narrowed to the bin that holds the last of them
    int32_t need = want - (lead + count - tail), in_bin = 0;
    const uint64_t range = hi - lo;
    int shift = range >> kBits ? 64 - kBits - __clzll((long long)range) : 0;
    for (;;) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = keys[i];
            if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        cluster.sync();
        // Thread t has the bins 4t .. 4t + 3 counted from the top.
        constexpr int kEach = kBins / kThreads;
        uint32_t v[kEach] = {};
        for (int r = 0; r < cl; ++r) {
            const uint32_t* x = cluster.map_shared_rank(&sh, r)->hist + kBins - kEach * (tid + 1);
            const uint4 y = *reinterpret_cast<const uint4*>(x);
            v[0] += y.w, v[1] += y.z, v[2] += y.y, v[3] += y.x;
        }
        static_assert(kEach == 4, "one 16-byte load");
        int32_t sum = v[0] + v[1] + v[2] + v[3], incl = sum;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += y;
        }
        if (lane == 31) ired[warp] = incl;
        if (tid == 0) found[0] = 0, found[1] = 0, found[2] = 0;
        __syncthreads();
        int32_t above = incl - sum;
        for (int w = 0; w < warp; ++w) above += ired[w];
        if (above < need && above + sum >= need) {
            int k = 0;
            while (above + (int32_t)v[k] < need) above += v[k++];
            found[0] = kBins - 1 - kEach * tid - k;
            found[1] = above;
            found[2] = v[k];
        }
        cluster.sync();  // the bins have been read, by all
        need -= found[1];
        in_bin = found[2];
        lo += (uint64_t)found[0] << shift;
        hi = lo + ((1ull << shift) - 1);
        if (in_bin <= need || shift == 0) break;
        for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
        shift = max(0, shift - kBits);
        __syncthreads();
    }
    // Taken: kept pages, keys above hi, and of those in [lo, hi] all, or (equal keys then) the first `need`.
    const bool ties = in_bin > need;
    int32_t n_above = 0, n_equal = 0;
    for (int i = tid; i < n; i += kThreads) {
        const bool kept = p0 + i < lead || p0 + i >= tail;
        n_above += kept || keys[i] > hi;
        n_equal += !kept && keys[i] >= lo && keys[i] <= hi;
    }
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    n_equal = __reduce_add_sync(0xffffffffu, n_equal);
    if (lane == 0) ired[warp] = n_above, ired[kWarps + warp] = n_equal;
    __syncthreads();
    if (tid == 0) {
        n_above = n_equal = 0;
        for (int w = 0; w < kWarps; ++w) n_above += ired[w], n_equal += ired[kWarps + w];
        sh.above = n_above, sh.equal = n_equal;
    }
    cluster.sync();
    int32_t at_out = 0, eq_before = 0;  // results and equal keys of the blocks before this one
    for (int r = 0; r < rank; ++r) {
        const Shared* x = cluster.map_shared_rank(&sh, r);
        const int32_t e = x->equal;
        at_out += x->above + (ties ? max(0, min(e, need - eq_before)) : e);
        eq_before += e;
    }
    cluster.sync();  // nobody reads this block's memory from here on
    for (int32_t base = 0; base < n; base += kThreads) {
        const int32_t i = base + tid;
        const bool kept = i < n && (p0 + i < lead || p0 + i >= tail);
        const uint64_t k = i < n ? keys[i] : 0;
        const bool sure = kept || (i < n && k > hi), equal = i < n && !kept && k >= lo && k <= hi;
        const uint32_t se = __ballot_sync(0xffffffffu, sure), ee = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) ired[warp] = __popc(se), ired[kWarps + warp] = __popc(ee);
        __syncthreads();
        int32_t eq = eq_before, sures = 0, eq_all = 0, sures_all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) eq += eq_all, sures = sures_all;
            eq_all += ired[kWarps + w];
            sures_all += ired[w];
        }
        const uint32_t lt = (1u << lane) - 1;
        const int32_t eq_mine = eq + __popc(ee & lt);  // equal keys before this page
        const int32_t take = ties ? need : INT32_MAX;
        if (sure || (equal && eq_mine < take)) {
            const int32_t pos = at_out + sures + __popc(se & lt) + min(eq_mine, take) - min(eq_before, take);
            if (pos < n_select) out[pos] = p0 + i;
        }
        at_out += sures_all + min(eq_before + eq_all, take) - min(eq_before, take);
        eq_before += eq_all;
        __syncthreads();
    }
}

template <typename T, int LP, int NC>
cudaError_t launch(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds, const int32_t* table,
                   const int32_t* seq_len, int32_t n_select, int32_t keep_first, int32_t keep_last, int32_t* pages,
                   int32_t* status, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // Blocks a row: as many as its scores need room for, then until the blocks fill the GPU twice, while each keeps
    // 128 pages.
    const int64_t rows = (int64_t)m.n_seqs * m.hkv;
    int cl = 1;
    while (cl < kMaxCluster && (m.max_pages > (int64_t)cl * kMaxShare ||
                                (rows * cl < 2 * sms && m.max_pages > (int64_t)cl * 2 * 128)))
        cl *= 2;
    auto kern = select_kernel<T, LP, NC>;
    const size_t smem = sizeof(uint64_t) * ((m.max_pages + cl - 1) / cl);
    static SmemGrants granted;
    e = allow_smem((const void*)kern, sizeof(uint64_t) * kMaxShare, granted);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return note_error(cudaLaunchKernelEx(&cfg, kern, m, (const T*)q, q_stride, (const T*)k_bounds, table, seq_len,
                                         n_select, keep_first, keep_last, pages, status, (int32_t)cl),
                      "paged select");
}

}  // namespace

cudaError_t launch_paged_select(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds,
                                const int32_t* table, const int32_t* seq_len, int32_t n_select, int32_t keep_first,
                                int32_t keep_last, int32_t* pages, int32_t* status, cudaStream_t st) {
#define SPLITKV_SELECT(T, LP, NC) \
    launch<T, LP, NC>(m, q, q_stride, k_bounds, table, seq_len, n_select, keep_first, keep_last, pages, status, st)
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
