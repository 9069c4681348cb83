// Keys and values of new tokens into a paged cache, rotary positions applied on the way.
#include <math.h>

#include "paged.cuh"

namespace splitkv {
namespace {

// Where token i goes. Padding and tokens out of range have page -1; the order is checked against the token
// before it that is not padding.
__device__ TokenPlace token_place(const PagedMeta& m, const AppendArgs& a, int64_t i, int32_t* status) {
    TokenPlace t{__ldg(a.token_seq + i), __ldg(a.token_pos + i), -1};
    if (t.seq < 0) return t;
    if (t.seq >= m.n_seqs || t.pos < 0 || t.pos >= (int64_t)m.max_pages * m.page ||
        (a.rope && t.pos >= a.rope_len)) {
        raise_status(status, SPLITKV_DEV_BAD_TOKEN);
        return t;
    }
    t.page = paged_page(m, a.table + t.seq * m.table_stride, t.pos >> m.page_shift, status);
    return t;
}

// Channel i of a row, rotated at the row of cosines and sines `cs` (null: as it is).
template <typename T>
__device__ T rotated(const AppendArgs& a, const T* x, int32_t i, const float* cs) {
    const int32_t half = a.rope_dim / 2;
    if (!cs || i >= a.rope_dim) return x[i];
    const int32_t pair = a.interleaved ? i / 2 : i % half;
    const bool second = a.interleaved ? i & 1 : i >= half;
    const float c = cs[pair], s = cs[half + pair];
    const float u = to_f32<T>(x[a.interleaved ? 2 * pair : pair]);
    const float w = to_f32<T>(x[a.interleaved ? 2 * pair + 1 : pair + half]);
    return from_f32<T>(second ? fmaf(w, c, u * s) : fmaf(u, c, -(w * s)));
}

// One block per token: queries, keys and values.
template <typename T>
__global__ void __launch_bounds__(128) append_rows_kernel(PagedMeta m, AppendArgs a, int32_t* status) {
    if (status_bad(status)) return;
    const int64_t i = blockIdx.x;
    const TokenPlace t = token_place(m, a, i, status);
    if (t.seq >= 0 && threadIdx.x == 0) {
        int64_t p = i - 1;
        while (p >= 0 && a.token_seq[p] < 0) --p;
        if (p >= 0 && (a.token_seq[p] > t.seq || (a.token_seq[p] == t.seq && a.token_pos[p] >= t.pos)))
            raise_status(status, SPLITKV_DEV_TOKEN_ORDER);
    }
    const float* cs = a.rope && t.page >= 0 ? a.rope + (int64_t)t.pos * a.rope_dim : nullptr;
    if (a.q)
        for (int32_t e = threadIdx.x; e < m.hq * m.d; e += 128) {
            const T* x = (const T*)a.q + i * a.q_stride + e / m.d * m.d;
            ((T*)a.q_out)[i * m.hq * m.d + e] = rotated<T>(a, x, e % m.d, cs);
        }
    if (t.page < 0) return;
    for (int32_t e = threadIdx.x; e < m.hkv * m.d; e += 128) {
        const int32_t g = e / m.d, c = e % m.d;
        const int64_t at = paged_row(m, t.page, g, t.pos & (m.page - 1)) + c;
        ((T*)a.k_cache)[at] = rotated<T>(a, (const T*)a.k + i * a.k_stride + g * m.d, c, cs);
        ((T*)a.v_cache)[at] = ((const T*)a.v)[i * a.v_stride + e];
    }
}

// One block per token: the bounds of its page, if no later token of the call writes the same page.
template <typename T>
__global__ void __launch_bounds__(128) append_bounds_kernel(PagedMeta m, AppendArgs a, int32_t* status) {
    if (status_bad(status)) return;
    const int64_t i = blockIdx.x;
    const TokenPlace t = token_place(m, a, i, status);
    if (t.page < 0) return;
    int64_t n = i + 1;
    while (n < a.n_tokens && a.token_seq[n] < 0) ++n;
    if (n < a.n_tokens && a.token_seq[n] == t.seq && a.token_pos[n] >> m.page_shift == t.pos >> m.page_shift) return;
    const int32_t last = t.pos & (m.page - 1);
    for (int32_t e = threadIdx.x; e < m.hkv * m.d; e += 128) {
        const int32_t g = e / m.d, c = e % m.d;
        float lo = INFINITY, hi = -INFINITY;
        for (int32_t off = 0; off <= last; ++off) {
            const float x = to_f32<T>(((const T*)a.k_cache)[paged_row(m, t.page, g, off) + c]);
            lo = fminf(lo, x);
            hi = fmaxf(hi, x);
        }
        T* dst = (T*)a.k_bounds + ((t.page * m.hkv + g) * 2) * m.d + c;
        dst[0] = from_f32<T>(lo);
        dst[m.d] = from_f32<T>(hi);
    }
}

template <typename T>
cudaError_t launch(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st) {
    append_rows_kernel<T><<<(unsigned)a.n_tokens, 128, 0, st>>>(m, a, status);
    if (a.k_bounds) append_bounds_kernel<T><<<(unsigned)a.n_tokens, 128, 0, st>>>(m, a, status);
    return note_error(cudaGetLastError(), "paged append");
}

}  // namespace

cudaError_t launch_paged_append(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st) {
    return m.dtype == SPLITKV_BF16 ? launch<__nv_bfloat16>(m, a, status, st) : launch<float>(m, a, status, st);
}

}  // namespace splitkv
