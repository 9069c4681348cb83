// Shared definitions of the paged-cache operators (append, one-token decode attention, page selection): the cache's
// geometry by value, row addressing and the internal launcher declarations.
#pragma once

#include <atomic>

#include "common.cuh"

namespace splitkv {

// Geometry of a paged cache, by value. Strides in elements; page_size is a power of two.
struct PagedMeta {
    int32_t hq, hkv, group, d;
    int32_t page, page_shift;   // positions per page, log2 of it
    int32_t max_pages;          // entries of a page-table row that may be read
    int32_t n_seqs;
    int64_t n_pages;            // pages of the cache
    int64_t table_stride;
    int64_t page_stride, head_stride, token_stride;
    float scale;
    int32_t dtype;
};

// The tokens of one append call.
struct AppendArgs {
    int64_t n_tokens;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token's first row to the next token's
    const float* rope;                     // [rope_len][rope_dim]: rope_dim/2 cosines, then rope_dim/2 sines; or null
    int32_t rope_dim, interleaved;
    int64_t rope_len;
    const int32_t *table, *token_seq, *token_pos;
    void *q_out, *k_cache, *v_cache, *k_bounds;
};

// A token's place in the cache. page < 0: not to be written (padding, or a reason already in the status word).
struct TokenPlace {
    int32_t seq, pos;
    int64_t page;
};

cudaError_t launch_paged_append(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st);

cudaError_t launch_paged_decode(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, const int32_t* table, const int32_t* seq_len,
                                const int32_t* pages, int32_t n_select, void* o, float* lse, int32_t* status, void* ws,
                                cudaStream_t st);
size_t paged_decode_workspace(const PagedMeta& m);
// The most units of work (16 positions at a kv head and 8 query rows) that one sequence may have. A launch counts its
// sequences' in 31 bits; a call makes as many launches as that takes.
int64_t paged_decode_units(const PagedMeta& m);

cudaError_t launch_paged_select(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_bounds,
                                const int32_t* table, const int32_t* seq_len, int32_t n_select, int32_t keep_first,
                                int32_t keep_last, int32_t* pages, int32_t* status, void* ws, cudaStream_t st);
size_t paged_select_workspace(const PagedMeta& m);
constexpr int32_t kMaxSelectPages = SPLITKV_PAGED_MAX_SELECT_PAGES;

// SMs of the current device, and the opt-in to the `most` bytes of dynamic shared memory that a kernel is ever launched
// with (`granted`: a static of the caller's for that kernel). Both are asked of the runtime once per device.
cudaError_t sm_count(int* sms);
using SmemGrants = std::atomic<bool>[kMaxDevices];
cudaError_t allow_smem(const void* kernel, size_t most, SmemGrants& granted);

// Launch in which the kernel may be placed on the SMs while the one before it in the stream drains. Every thread of it
// calls after_previous(), which waits until that one has completed and its writes are seen, before it touches memory. That
// holds for the second kernel of a call too: that the first one has waited says nothing of what the second one sees. Hides
// the launch's own latency (2 us of every call), felt where a call takes ten.
// So what these kernels read may be written while they are resident: they read it with coherent loads behind the wait, not
// through the read-only path (ld.global.nc, __ldg, const __restrict__ parameters), which asks for data that does not change
// while the kernel lives and which the compiler may move ahead of the wait.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Length of sequence b, or 0 (with the status bit) when it is not in [0, max_pages * page].
__device__ __forceinline__ int32_t paged_len(const PagedMeta& m, const int32_t* seq_len, int32_t b, int32_t* status) {
    const int32_t n = seq_len[b];
    if (n < 0 || n > (int64_t)m.max_pages * m.page) {
        raise_status(status, SPLITKV_DEV_BAD_LENGTH);
        return 0;
    }
    return n;
}

// Cache page behind entry `e` of a page-table row, or -1 (with the status bit) when it is out of range.
__device__ __forceinline__ int32_t paged_page(const PagedMeta& m, const int32_t* row, int32_t e, int32_t* status) {
    const int32_t p = row[e];
    if (p < 0 || p >= m.n_pages) {
        raise_status(status, SPLITKV_DEV_BAD_PAGE);
        return -1;
    }
    return p;
}

__device__ __forceinline__ int64_t paged_row(const PagedMeta& m, int64_t page, int32_t g, int32_t off) {
    return page * m.page_stride + g * m.head_stride + off * m.token_stride;
}

// 16 bytes that are read once, or zeros. Predicated rather than branched around (a branch per load cost more than the
// load), and volatile: the loads stay where they are issued, ahead of the work that hides them (the compiler would move
// them down to their use).
__device__ __forceinline__ uint4 ldg_stream_if(const void* p, bool in) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(p), "r"((int)in));
    return r;
}

}  // namespace splitkv
