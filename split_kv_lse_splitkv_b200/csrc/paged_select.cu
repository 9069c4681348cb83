// Selection of the pages that a sequence's new token reads, by a bound on its scores.
#include <math.h>

#include "paged.cuh"

namespace splitkv {
namespace {

constexpr int kSelThreads = 256;

// The order of the scores as unsigned integers: larger score, larger key. NaN: below every number.
__device__ __forceinline__ uint64_t score_key(double s) {
    if (s != s) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);  // -0 ranks as 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

template <typename T>
__device__ double page_score(const PagedMeta& m, const T* q, int64_t q_stride, const T* bounds, int32_t b, int32_t g,
                             int64_t page) {
    const T* lo = bounds + (page * m.hkv + g) * 2 * m.d;
    double s = 0.0;
    for (int i = 0; i < m.d; ++i) {
        double up = 0.0, down = 0.0;
        for (int h = g * m.group; h < (g + 1) * m.group; ++h) {
            const double x = to_f32<T>(q[b * q_stride + (int64_t)h * m.d + i]);
            up += x > 0.0 ? x : 0.0;
            down += x < 0.0 ? x : 0.0;
        }
        s += up * to_f32<T>(lo[m.d + i]) + down * to_f32<T>(lo[i]);
    }
    return s;
}

// One block per (sequence, kv head). Finds the key of the n-th page by bits, from the top, recomputing the scores.
template <typename T>
__global__ void __launch_bounds__(kSelThreads) select_simple_kernel(PagedMeta m, const T* __restrict__ q,
                                                                    int64_t q_stride, const T* __restrict__ bounds,
                                                                    const int32_t* __restrict__ table,
                                                                    const int32_t* __restrict__ seq_len,
                                                                    int32_t n_select, int32_t keep_first,
                                                                    int32_t keep_last, int32_t* __restrict__ pages,
                                                                    int32_t* status) {
    extern __shared__ uint64_t keys[];
    __shared__ int32_t total;
    if (status_bad(status)) return;
    const int32_t b = blockIdx.x / m.hkv, g = blockIdx.x % m.hkv, tid = threadIdx.x;
    const int32_t len = paged_len(m, seq_len, b, status);
    const int32_t count = (len + m.page - 1) >> m.page_shift;
    int32_t* out = pages + ((int64_t)b * m.hkv + g) * n_select;
    auto key_of = [&](int32_t p) -> uint64_t {
        if (p < keep_first || p >= count - keep_last) return ~0ull;
        const int32_t page = paged_page(m, table + b * m.table_stride, p, status);
        return page < 0 ? 0 : score_key(page_score(m, q, q_stride, bounds, b, g, page));
    };
    auto sum = [&](int32_t x) {
        __syncthreads();
        if (tid == 0) total = 0;
        __syncthreads();
        atomicAdd(&total, x);
        __syncthreads();
        return total;
    };
    // Largest key t with at least min(n_select, count) keys >= t.
    const int32_t want = min(n_select, count);
    uint64_t t = 0;
    if (count > n_select)
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t probe = t | 1ull << bit;
            int32_t mine = 0;
            for (int32_t p = tid; p < count; p += kSelThreads) mine += key_of(p) >= probe;
            if (sum(mine) >= want) t = probe;
        }
    int32_t mine = 0;
    if (count > n_select)
        for (int32_t p = tid; p < count; p += kSelThreads) mine += key_of(p) > t;
    int32_t equal = want - sum(mine);  // how many pages with the key t itself come in, lowest first
    if (tid == 0) {
        int32_t n = 0;
        for (int32_t p = 0; p < count && n < want; ++p) {
            const uint64_t k = count > n_select ? key_of(p) : 1;
            if (count <= n_select || k > t || (k == t && equal-- > 0)) out[n++] = p;
        }
        for (; n < n_select; ++n) out[n] = -1;
    }
}

}  // namespace

cudaError_t launch_paged_select(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds,
                                const int32_t* table, const int32_t* seq_len, int32_t n_select, int32_t keep_first,
                                int32_t keep_last, int32_t* pages, int32_t* status, cudaStream_t st) {
    const int grid = m.n_seqs * m.hkv;
    if (m.dtype == SPLITKV_BF16)
        select_simple_kernel<__nv_bfloat16><<<grid, kSelThreads, 0, st>>>(
            m, (const __nv_bfloat16*)q, q_stride, (const __nv_bfloat16*)k_bounds, table, seq_len, n_select, keep_first,
            keep_last, pages, status);
    else
        select_simple_kernel<float><<<grid, kSelThreads, 0, st>>>(m, (const float*)q, q_stride,
                                                                  (const float*)k_bounds, table, seq_len, n_select,
                                                                  keep_first, keep_last, pages, status);
    return note_error(cudaGetLastError(), "paged select");
}

}  // namespace splitkv
