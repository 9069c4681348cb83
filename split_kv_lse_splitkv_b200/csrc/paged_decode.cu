// Attention of one new token of each sequence over a paged key-value cache.
#include <math.h>

#include "paged.cuh"

namespace splitkv {
namespace {

// One warp per (sequence, query head): an online softmax over the keys one at a time, lanes over the channels.
template <typename T>
__global__ void __launch_bounds__(32) decode_simple_kernel(PagedMeta m, const T* __restrict__ q, int64_t q_stride,
                                                          const T* __restrict__ kc, const T* __restrict__ vc,
                                                          const int32_t* __restrict__ table,
                                                          const int32_t* __restrict__ seq_len,
                                                          const int32_t* __restrict__ pages, int32_t n_select,
                                                          T* __restrict__ o, float* __restrict__ lse,
                                                          int32_t* status) {
    if (status_bad(status)) return;
    const int32_t b = blockIdx.x / m.hq, h = blockIdx.x % m.hq, g = h / m.group, lane = threadIdx.x;
    const int32_t len = paged_len(m, seq_len, b, status);
    const int32_t count = (len + m.page - 1) >> m.page_shift;
    const int32_t* row = table + b * m.table_stride;
    const int32_t* list = pages ? pages + ((int64_t)b * m.hkv + g) * n_select : nullptr;
    float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int u = 0; u < 4; ++u)
        qv[u] = lane + 32 * u < m.d ? to_f32<T>(q[b * q_stride + (int64_t)h * m.d + lane + 32 * u]) * m.scale : 0.f;
    float mx = -INFINITY, l = 0.f;
    int32_t before = -1;
    const int32_t n = list ? n_select : count;
    for (int32_t e = 0; e < n; ++e) {
        int32_t entry = e;
        if (list) {
            entry = list[e];
            if (entry < -1 || entry >= count || (entry >= 0 && (entry <= before || (e > 0 && list[e - 1] < 0)))) {
                raise_status(status, SPLITKV_DEV_BAD_PAGE);
                break;
            }
            if (entry < 0) continue;
            before = entry;
        }
        const int32_t page = paged_page(m, row, entry, status);
        if (page < 0) continue;
        const int32_t here = min(m.page, len - (entry << m.page_shift));
        for (int32_t off = 0; off < here; ++off) {
            const int64_t at = paged_row(m, page, g, off);
            float s = 0.f;
            for (int u = 0; u < 4; ++u)
                if (lane + 32 * u < m.d) s += qv[u] * to_f32<T>(kc[at + lane + 32 * u]);
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            const float top = fmaxf(mx, s);
            if (top == -INFINITY) continue;
            const float fix = expf(mx - top), p = expf(s - top);
            l = l * fix + p;
            for (int u = 0; u < 4; ++u)
                if (lane + 32 * u < m.d) acc[u] = acc[u] * fix + p * to_f32<T>(vc[at + lane + 32 * u]);
            mx = top;
        }
    }
    const int64_t out = (int64_t)b * m.hq + h;
    for (int u = 0; u < 4; ++u)
        if (lane + 32 * u < m.d) o[out * m.d + lane + 32 * u] = from_f32<T>(l > 0.f ? acc[u] / l : 0.f);
    if (lane == 0) lse[out] = l > 0.f ? mx + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_decode_workspace(const PagedMeta& m) { return 256; }

cudaError_t launch_paged_decode(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, const int32_t* table, const int32_t* seq_len,
                                const int32_t* pages, int32_t n_select, void* o, float* lse, int32_t* status, void* ws,
                                cudaStream_t st) {
    const int grid = m.n_seqs * m.hq;
    if (m.dtype == SPLITKV_BF16)
        decode_simple_kernel<__nv_bfloat16><<<grid, 32, 0, st>>>(
            m, (const __nv_bfloat16*)q, q_stride, (const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache, table,
            seq_len, pages, n_select, (__nv_bfloat16*)o, lse, status);
    else
        decode_simple_kernel<float><<<grid, 32, 0, st>>>(m, (const float*)q, q_stride, (const float*)k_cache,
                                                         (const float*)v_cache, table, seq_len, pages, n_select,
                                                         (float*)o, lse, status);
    return note_error(cudaGetLastError(), "paged decode");
}

}  // namespace splitkv
