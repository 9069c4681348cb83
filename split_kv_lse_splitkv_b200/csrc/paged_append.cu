// Keys and values of new tokens into a paged cache, rotary positions applied on the way.
//
// Bound by the bytes of the rows in and out. A lane holds two pieces (16 bytes) of a row whose channels are each other's
// partners in the rotation, so it rotates them in registers; a warp takes several rows at once. The bounds over the keys of
// a page that is written are one warp's work (or one block's), the one that finds the call's first token in that page: no
// two write one page's bounds. Few tokens: rows and bounds in one launch, the new keys turned a second time for their bounds
// so that nothing waits. Many: rows first, then the bounds from the keys as the cache holds them, in L2.
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace splitkv {
namespace {

// 128 threads a block 140 us, 256 143, 512 149 (35k tokens, 32/4 heads).
constexpr int kThreads = 128, kWarps = kThreads / 32;

// Where token i goes. Padding and tokens out of range have page -1.
__device__ TokenPlace token_place(const PagedMeta& m, const AppendArgs& a, int64_t i, int32_t* status) {
    TokenPlace t{a.token_seq[i], a.token_pos[i], -1};
    if (t.seq < 0) return t;
    if (t.seq >= m.n_seqs || t.pos < 0 || t.pos >= (int64_t)m.max_pages * m.page ||
        (a.rope && t.pos >= a.rope_len)) {
        raise_status(status, SPLITKV_DEV_BAD_TOKEN);
        return t;
    }
    t.page = paged_page(m, a.table + t.seq * m.table_stride, t.pos >> m.page_shift, status);
    return t;
}

// The nearest token before i (kAfter: after i) that is not padding, or -1, on a whole warp with the same i in each lane: 256
// tokens a step, because a padded batch has long runs of padding (one thread, token by token: 8 rows padded to 4096, a third
// of them tokens, 32/4 heads, d 128: 400 us; so: 108). Not inlined: it is rarely called, and the callers need the registers.
template <bool kAfter>
__device__ __noinline__ int64_t token_beside(const AppendArgs& a, int64_t i, int lane) {
    constexpr int kLook = 8;
    for (int64_t base = 1; kAfter ? i + base < a.n_tokens : i - base >= 0; base += kLook * 32) {
        uint32_t real[kLook];
#pragma unroll
        for (int u = 0; u < kLook; ++u) {
            const int64_t p = kAfter ? i + base + u * 32 + lane : i - base - u * 32 - lane;
            real[u] = p >= 0 && p < a.n_tokens && a.token_seq[p] >= 0;
        }
#pragma unroll
        for (int u = 0; u < kLook; ++u) {
            const uint32_t found = __ballot_sync(0xffffffffu, real[u]);
            if (found) return kAfter ? i + base + u * 32 + __ffs(found) - 1 : i - base - u * 32 - __ffs(found) + 1;
        }
    }
    return -1;
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

// ---- any rope_dim: channels one by one. One block per token: queries, keys and values.
// Both kernels leave as whole blocks: other blocks raise the status word meanwhile, and token_beside() needs all lanes.
template <typename T>
__global__ void __launch_bounds__(128) append_channels_kernel(PagedMeta m, AppendArgs a, int32_t* status) {
    if (__syncthreads_or(status_bad(status))) return;
    const int64_t i = blockIdx.x;
    const TokenPlace t = token_place(m, a, i, status);
    if (t.seq >= 0 && threadIdx.x < 32) {
        const int64_t p = token_beside<false>(a, i, threadIdx.x);
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
__global__ void __launch_bounds__(128) append_channels_bounds_kernel(PagedMeta m, AppendArgs a, int32_t* status) {
    if (__syncthreads_or(status_bad(status))) return;
    const int64_t i = blockIdx.x;
    const TokenPlace t = token_place(m, a, i, status);
    if (t.page < 0) return;
    const int64_t n = token_beside<true>(a, i, threadIdx.x & 31);
    if (n >= 0 && a.token_seq[n] == t.seq && a.token_pos[n] >> m.page_shift == t.pos >> m.page_shift) return;
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

// ---- pieces of 16 bytes, or of 8: half of rope_dim has to be whole pieces

// What is loaded and stored as one, and arithmetic on it.
__device__ __forceinline__ void load_if(uint4& x, const void* p, bool in) { x = ldg_stream_if(p, in); }
__device__ __forceinline__ void load_if(uint2& x, const void* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
        "@p ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n\t}"
        : "=&r"(x.x), "=&r"(x.y)
        : "l"(p), "r"((int)in));
}
template <typename Type>
struct Word;  // 32 bits
template <>
struct Word<__nv_bfloat16> {
    static constexpr int kN = 2;
    static __device__ __forceinline__ void unpack(uint32_t w, float* f) {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(const float* f) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f[1]), "f"(f[0]));
        return w;
    }
    template <bool kMax>
    static __device__ __forceinline__ uint32_t best(uint32_t x, uint32_t y) {
        const __nv_bfloat162 u = *reinterpret_cast<__nv_bfloat162*>(&x), v = *reinterpret_cast<__nv_bfloat162*>(&y);
        const __nv_bfloat162 r = kMax ? __hmax2(u, v) : __hmin2(u, v);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static constexpr uint32_t kInf = 0x7f807f80u, kNegInf = 0xff80ff80u;
};
template <>
struct Word<float> {
    static constexpr int kN = 1;
    static __device__ __forceinline__ void unpack(uint32_t w, float* f) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t pack(const float* f) { return __float_as_uint(f[0]); }
    template <bool kMax>
    static __device__ __forceinline__ uint32_t best(uint32_t x, uint32_t y) {
        const float u = __uint_as_float(x), v = __uint_as_float(y);
        return __float_as_uint(kMax ? fmaxf(u, v) : fminf(u, v));
    }
    static constexpr uint32_t kInf = 0x7f800000u, kNegInf = 0xff800000u;
};
__device__ __forceinline__ uint32_t& word(uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }
__device__ __forceinline__ uint32_t& word(uint2& x, int i) { return i == 0 ? x.x : x.y; }
__device__ __forceinline__ uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }
__device__ __forceinline__ uint32_t word(const uint2& x, int i) { return i == 0 ? x.x : x.y; }

template <typename Type, typename Of>
struct Vec {
    using T = Type;
    using Piece = Of;
    using W = Word<T>;
    static constexpr int kWords = sizeof(Piece) / 4, kN = kWords * W::kN;
    static __device__ __forceinline__ void unpack(const Piece& x, float (&f)[kN]) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) W::unpack(word(x, i), f + i * W::kN);
    }
    static __device__ __forceinline__ Piece pack(const float (&f)[kN]) {
        Piece x;
#pragma unroll
        for (int i = 0; i < kWords; ++i) word(x, i) = W::pack(f + i * W::kN);
        return x;
    }
    static __device__ __forceinline__ Piece all(uint32_t w) {
        Piece x;
#pragma unroll
        for (int i = 0; i < kWords; ++i) word(x, i) = w;
        return x;
    }
};

template <typename V, bool kMax>
__device__ __forceinline__ void take(typename V::Piece& x, const typename V::Piece& y) {
#pragma unroll
    for (int i = 0; i < V::kWords; ++i) word(x, i) = V::W::template best<kMax>(word(x, i), word(y, i));
}

// How a row of d channels lies over lanes: `per_row` lanes a row, two pieces a lane.
struct Lanes {
    int per_row, rows;  // rows: how many a warp takes at once
    int row, a, b;      // this lane's row (>= rows: none), first channels of its pieces (b < 0: only one)
    int pair;           // first angle of its pairs, or -1: not rotated
};

template <typename V>
__device__ __forceinline__ Lanes lanes_of(int d, int rope_dim, int interleaved, int lane) {
    constexpr int kN = V::kN;
    const int turned = rope_dim / 2 / kN, rest = (d - rope_dim) / kN;
    Lanes x;
    x.per_row = turned + (rest + 1) / 2;
    x.rows = 32 / x.per_row;
    x.row = lane / x.per_row;
    const int j = lane - x.row * x.per_row;
    if (j < turned) {
        x.a = interleaved ? 2 * j * kN : j * kN;
        x.b = interleaved ? x.a + kN : rope_dim / 2 + x.a;
        x.pair = j * kN;
    } else {
        x.a = rope_dim + 2 * (j - turned) * kN;
        x.b = x.a + kN < d ? x.a + kN : -1;
        x.pair = -1;
    }
    return x;
}

template <typename V>
struct Angles {
    using Piece = typename V::Piece;
    float c[V::kN], s[V::kN];
    __device__ __forceinline__ void load(const float* row, int half, int pair) {
#pragma unroll
        for (int i = 0; i < V::kN; i += 4) {
            if constexpr (V::kN >= 4) {
                const float4 x = *reinterpret_cast<const float4*>(row + pair + i);
                const float4 y = *reinterpret_cast<const float4*>(row + half + pair + i);
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(row + pair);
                const float2 y = *reinterpret_cast<const float2*>(row + half + pair);
                c[0] = x.x, c[1] = x.y, s[0] = y.x, s[1] = y.y;
            }
        }
    }
    // (x c - y s, y c + x s) for each pair (x, y), in float32, rounded once to the type.
    __device__ __forceinline__ void turn(Piece& a, Piece& b, int interleaved) const {
        constexpr int kN = V::kN;
        float x[kN], y[kN], u[kN], w[kN];
        V::unpack(a, x);
        V::unpack(b, y);
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) {
                u[2 * i] = fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i]));
                u[2 * i + 1] = fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]);
                w[2 * i] = fmaf(y[2 * i], c[kN / 2 + i], -(y[2 * i + 1] * s[kN / 2 + i]));
                w[2 * i + 1] = fmaf(y[2 * i + 1], c[kN / 2 + i], y[2 * i] * s[kN / 2 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                u[i] = fmaf(x[i], c[i], -(y[i] * s[i]));
                w[i] = fmaf(y[i], c[i], x[i] * s[i]);
            }
        }
        a = V::pack(u);
        b = V::pack(w);
    }
};

// Which of the `slice` <= 32 tokens from i0 on (a lane each) are the first of the call in their page. `report`: say what is
// wrong with them, their order included, in the status word.
__device__ __forceinline__ uint32_t page_firsts(const PagedMeta& m, const AppendArgs& a, int64_t i0, int32_t slice,
                                                int lane, bool report, int32_t* status) {
    if (i0 >= a.n_tokens) return 0;
    const int64_t i = i0 + lane;
    const bool mine = lane < slice && i < a.n_tokens;
    const int32_t seq = mine ? a.token_seq[i] : -1, pos = mine ? a.token_pos[i] : 0;
    int32_t before = i0 > 0 ? a.token_seq[i0 - 1] : -1, before_pos = i0 > 0 ? a.token_pos[i0 - 1] : -1;
    const uint32_t real = __ballot_sync(0xffffffffu, seq >= 0), below = real & ((1u << lane) - 1);
    if (!real) return 0;
    if (i0 > 0 && before < 0) {  // padding before the slice
        const int64_t p = token_beside<false>(a, i0 - 1, lane);
        if (p >= 0) before = a.token_seq[p], before_pos = a.token_pos[p];
    }
    const int from = below ? 31 - __clz(below) : 0;
    const int32_t s = __shfl_sync(0xffffffffu, seq, from), p = __shfl_sync(0xffffffffu, pos, from);
    if (below) before = s, before_pos = p;
    bool first = seq >= 0;
    if (first) {
        if (report && (before > seq || (before == seq && before_pos >= pos))) raise_status(status, SPLITKV_DEV_TOKEN_ORDER);
        if (seq >= m.n_seqs || pos < 0 || pos >= (int64_t)m.max_pages * m.page || (a.rope && pos >= a.rope_len)) {
            if (report) raise_status(status, SPLITKV_DEV_BAD_TOKEN);
            first = false;
        } else if (before == seq && before_pos >= 0 && before_pos >> m.page_shift == pos >> m.page_shift) {
            first = false;
        }
    }
    return __ballot_sync(0xffffffffu, first);
}

// Rows by themselves. A unit is `most` rows: that many heads of one token, or all heads of several tokens where they are
// few. A warp has a unit of queries, or one of keys and the same one of values.
struct Units {
    int32_t heads, tokens;  // of a unit
    int32_t per_token;      // units that a token's heads take
    __host__ __device__ Units(int32_t all, int32_t most)
        : heads(all < most ? all : most), tokens(most / heads), per_token((all + heads - 1) / heads) {}
    __host__ __device__ int64_t of(int64_t n) const { return (n + tokens - 1) / tokens * per_token; }
};

template <typename V>
__device__ __forceinline__ void append_rows(const PagedMeta& m, const AppendArgs& a, int64_t unit, int lane, int32_t* status) {
    using T = typename V::T;
    using Piece = typename V::Piece;
    const Lanes L = lanes_of<V>(m.d, a.rope_dim, a.interleaved, lane);
    const Units Q(m.hq, 4 * L.rows), KV(m.hkv, 2 * L.rows);
    const int64_t q_units = a.q ? Q.of(a.n_tokens) : 0;
    const bool queries = unit < q_units;
    const Units U = queries ? Q : KV;
    if (!queries) unit -= q_units;
    const int64_t i0 = unit / U.per_token * U.tokens;
    const int32_t h0 = (int32_t)(unit % U.per_token) * U.heads;
    // Row x of the unit: token i0 + x / heads, head h0 + x % heads; a lane has rows L.row + k * L.rows.
    auto row = [&](int k, int64_t& i, int32_t& h) {
        const int32_t x = L.row + k * L.rows, t = U.tokens == 1 ? x >= U.heads : x / U.heads;
        i = i0 + t, h = h0 + x - t * U.heads;
        return L.row < L.rows && t < U.tokens && i < a.n_tokens && h < (queries ? m.hq : m.hkv);
    };
    Angles<V> ang;
    int64_t i[2];
    int32_t h[2];
    bool in[2];
    Piece x[2], y[2];
    if (queries) {
        int64_t now = -1;  // the token whose angles are at hand
        bool turn = false;
        for (int step = 0; step < 4; step += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                in[k] = row(step + k, i[k], h[k]);
                const T* src = (const T*)a.q + i[k] * a.q_stride + (int64_t)h[k] * m.d;
                load_if(x[k], src + L.a, in[k]);
                load_if(y[k], src + L.b, in[k] && L.b >= 0);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!in[k]) continue;
                if (i[k] != now) {
                    now = i[k];
                    const int32_t seq = a.token_seq[now], pos = a.token_pos[now];
                    // A token that is out of range is reported with its keys; its queries pass as they are.
                    turn = L.pair >= 0 && seq >= 0 && pos >= 0 && pos < a.rope_len;
                    if (turn) ang.load(a.rope + (int64_t)pos * a.rope_dim, a.rope_dim / 2, L.pair);
                }
                if (turn) ang.turn(x[k], y[k], a.interleaved);
                T* dst = (T*)a.q_out + (i[k] * m.hq + h[k]) * m.d;
                *reinterpret_cast<Piece*>(dst + L.a) = x[k];
                if (L.b >= 0) *reinterpret_cast<Piece*>(dst + L.b) = y[k];
            }
        }
        return;
    }
    Piece z[2], w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        in[k] = row(k, i[k], h[k]);
        const T* src = (const T*)a.k + i[k] * a.k_stride + (int64_t)h[k] * m.d;
        load_if(x[k], src + L.a, in[k]);
        load_if(y[k], src + L.b, in[k] && L.b >= 0);
        src = (const T*)a.v + i[k] * a.v_stride + (int64_t)h[k] * m.d;
        load_if(z[k], src + L.a, in[k]);
        load_if(w[k], src + L.b, in[k] && L.b >= 0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!in[k]) continue;
        const TokenPlace t = token_place(m, a, i[k], status);
        if (t.page < 0) continue;
        if (L.pair >= 0) {
            ang.load(a.rope + (int64_t)t.pos * a.rope_dim, a.rope_dim / 2, L.pair);
            ang.turn(x[k], y[k], a.interleaved);
        }
        const int64_t at = paged_row(m, t.page, h[k], t.pos & (m.page - 1));
        T* dst = (T*)a.k_cache + at;
        *reinterpret_cast<Piece*>(dst + L.a) = x[k];
        if (L.b >= 0) *reinterpret_cast<Piece*>(dst + L.b) = y[k];
        dst = (T*)a.v_cache + at;
        *reinterpret_cast<Piece*>(dst + L.a) = z[k];
        if (L.b >= 0) *reinterpret_cast<Piece*>(dst + L.b) = w[k];
    }
}

// Many tokens, first launch: rows. (With the bounds in the same launch, the registers they take cost the rows' loads in
// flight: 35k tokens 144 to 165 us in one launch, 140 in two.) 8 blocks an SM leave 64 registers, where bf16 in 16-byte pieces
// spills 76 bytes; that costs nothing: 142 us, 7 blocks without spills 141, 6 blocks 149.
template <typename V>
__global__ void __launch_bounds__(kThreads, 8) append_rows_kernel(PagedMeta m, AppendArgs a, int32_t* status) {
    after_previous();
    if (status_bad(status)) return;
    append_rows<V>(m, a, (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), threadIdx.x & 31, status);
}

// Second launch: what is wrong with the tokens' order (looking at it beside the rows costs 4 us of 140), and, at one kv
// head, the bounds of the pages whose first token of the call is among a warp's `slice`, from L2.
template <typename T>
__global__ void __launch_bounds__(kThreads, 7) append_bounds_kernel(PagedMeta m, AppendArgs a, int32_t* status,
                                                                   int32_t slice) {
    using V = Vec<T, uint4>;
    const int lane = threadIdx.x & 31;
    const int32_t heads = a.k_bounds ? m.hkv : 1;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), i0 = unit / heads * slice;
    const int32_t g = (int32_t)(unit % heads);
    const Lanes L = lanes_of<V>(m.d, 0, 0, lane);
    after_previous();
    uint32_t firsts = page_firsts(m, a, i0, slice, lane, g == 0, status);
    if (!a.k_bounds) return;
    for (; firsts; firsts &= firsts - 1) {
        const int64_t i = i0 + __ffs(firsts) - 1;
        const int32_t seq = a.token_seq[i], entry = a.token_pos[i] >> m.page_shift;
        const int32_t page = paged_page(m, a.table + seq * m.table_stride, entry, status);
        int32_t last = 0;  // the last of the page's tokens: they go on to the first token of another page
        for (int64_t base = i;; base += 32) {
            const int64_t t = base + lane;
            const int32_t s = t < a.n_tokens ? a.token_seq[t] : INT32_MAX;
            const int32_t q = s >= 0 && s < INT32_MAX ? a.token_pos[t] : -1;
            const bool in = s == seq && q >= 0 && q >> m.page_shift == entry;
            const uint32_t stops = __ballot_sync(0xffffffffu, s >= 0 && !in);
            const int end = stops ? __ffs(stops) - 1 : 32;
            last = max(last, __reduce_max_sync(0xffffffffu, in && lane < end ? q & (m.page - 1) : 0));
            if (stops) break;
            if (!__any_sync(0xffffffffu, s >= 0)) {  // padding: on to what comes after it
                const int64_t n = token_beside<true>(a, base + 31, lane);
                if (n < 0) break;
                base = n - 32;
            }
        }
        if (page < 0 || __any_sync(0xffffffffu, status_bad(status))) continue;
        uint4 lo[2], hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            lo[x] = V::all(V::W::kInf);
            hi[x] = V::all(V::W::kNegInf);
        }
        const T* kc = (const T*)a.k_cache + paged_row(m, page, g, 0);
        constexpr int kAhead = 4;
        for (int32_t off0 = 0; off0 <= last; off0 += kAhead * L.rows) {
            uint4 x[kAhead], y[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t off = off0 + u * L.rows + L.row;
                const bool in = L.row < L.rows && off <= last;
                x[u] = ldg_stream_if(kc + off * m.token_stride + L.a, in);
                y[u] = ldg_stream_if(kc + off * m.token_stride + L.b, in && L.b >= 0);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (L.row >= L.rows || off0 + u * L.rows + L.row > last) continue;
                take<V, false>(lo[0], x[u]), take<V, true>(hi[0], x[u]);
                take<V, false>(lo[1], y[u]), take<V, true>(hi[1], y[u]);
            }
        }
        for (int r = 1; r < L.rows; ++r) {  // the lanes of the first row take the others'
            auto from = [&](const uint4& x) {
                const int l = (lane + r * L.per_row) & 31;
                return make_uint4(__shfl_sync(0xffffffffu, x.x, l), __shfl_sync(0xffffffffu, x.y, l),
                                  __shfl_sync(0xffffffffu, x.z, l), __shfl_sync(0xffffffffu, x.w, l));
            };
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint4 l = from(lo[x]), h = from(hi[x]);
                if (lane < L.per_row) take<V, false>(lo[x], l), take<V, true>(hi[x], h);
            }
        }
        if (L.row == 0) {
            T* dst = (T*)a.k_bounds + ((int64_t)page * m.hkv + g) * 2 * m.d;
            *reinterpret_cast<uint4*>(dst + L.a) = lo[0];
            *reinterpret_cast<uint4*>(dst + m.d + L.a) = hi[0];
            if (L.b >= 0) {
                *reinterpret_cast<uint4*>(dst + L.b) = lo[1];
                *reinterpret_cast<uint4*>(dst + m.d + L.b) = hi[1];
            }
        }
    }
}

// Few tokens, one launch. The bounds of page `page` at kv head g, its new tokens the call's from i on, on the warps of a block that share it (`split`
// of them, this one `sub`; all of them come here together) or on one. New keys are turned once more: so nothing waits for the
// rows to be written, and the keys are in L2 twice in a row.
template <typename V>
__device__ __forceinline__ void page_bounds(const PagedMeta& m, const AppendArgs& a, int64_t i, int32_t page, int32_t g,
                                            int32_t split, int32_t sub, int lane, typename V::Piece (*red)[32][4]) {
    using T = typename V::T;
    using Piece = typename V::Piece;
    const Lanes L = lanes_of<V>(m.d, a.rope_dim, a.interleaved, lane);
    const int32_t seq = a.token_seq[i], entry = a.token_pos[i] >> m.page_shift;
    Piece lo[2], hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) lo[x] = V::all(V::W::kInf), hi[x] = V::all(V::W::kNegInf);
    auto see = [&](const Piece& x, const Piece& y) {
        take<V, false>(lo[0], x), take<V, true>(hi[0], x);
        take<V, false>(lo[1], y), take<V, true>(hi[1], y);
    };
    // The page's tokens go on to the first token of another page.
    int32_t last = 0;
    uint32_t is_new = 0;  // bit b of lane l: position 32 l + b
    int32_t n_new = 0;
    for (int64_t base = i;; base += 32) {
        const int64_t t = base + lane;
        const int32_t s = t < a.n_tokens ? a.token_seq[t] : INT32_MAX;
        const int32_t q = s >= 0 && s < INT32_MAX ? a.token_pos[t] : -1;
        bool in = s == seq && q >= 0 && q >> m.page_shift == entry;
        const uint32_t stops = __ballot_sync(0xffffffffu, s >= 0 && !in);
        in &= lane < (stops ? __ffs(stops) - 1 : 32);
        const uint32_t tokens = __ballot_sync(0xffffffffu, in);
        const int32_t off = q & (m.page - 1);
        n_new += __popc(tokens);
        if (tokens) {
            const int32_t top = __reduce_max_sync(0xffffffffu, in ? off : 0);
            last = max(last, top);
            for (int32_t w = __reduce_min_sync(0xffffffffu, in ? off : INT32_MAX) >> 5; w <= top >> 5; ++w) {
                const uint32_t bits = __reduce_or_sync(0xffffffffu, in && off >> 5 == w ? 1u << (off & 31) : 0);
                if (lane == w) is_new |= bits;
            }
            const int32_t end = 32 - __clz(tokens);
            constexpr int kAhead = 2;
#pragma unroll 1
            for (int32_t r = sub * kAhead * L.rows; r < end; r += split * kAhead * L.rows) {
                Piece x[kAhead], y[kAhead];
                int32_t pos[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int32_t at = r + u * L.rows + L.row;
                    const bool mine = L.row < L.rows && at < end && (tokens >> at & 1);
                    pos[u] = __shfl_sync(0xffffffffu, q, at & 31);
                    if (!mine || (a.rope && pos[u] >= a.rope_len)) pos[u] = -1;
                    const T* src = (const T*)a.k + (base + at) * a.k_stride + (int64_t)g * m.d;
                    load_if(x[u], src + L.a, mine);
                    load_if(y[u], src + L.b, mine && L.b >= 0);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (pos[u] < 0) continue;
                    if (L.pair >= 0) {
                        Angles<V> ang;
                        ang.load(a.rope + (int64_t)pos[u] * a.rope_dim, a.rope_dim / 2, L.pair);
                        ang.turn(x[u], y[u], a.interleaved);
                    }
                    see(x[u], y[u]);
                }
            }
        }
        if (stops) break;
        if (!__any_sync(0xffffffffu, s >= 0)) {  // padding: on to what comes after it
            const int64_t n = token_beside<true>(a, base + 31, lane);
            if (n < 0) break;
            base = n - 32;
        }
    }
    if (n_new <= last) {  // keys that were there
        const T* kc = (const T*)a.k_cache + paged_row(m, page, g, 0);
        constexpr int kAhead = 4;
#pragma unroll 1
        for (int32_t off0 = sub * kAhead * L.rows; off0 < last; off0 += split * kAhead * L.rows) {
            Piece x[kAhead], y[kAhead];
            bool in[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t off = off0 + u * L.rows + L.row;
                const uint32_t bits = __shfl_sync(0xffffffffu, is_new, off >> 5 & 31);
                in[u] = L.row < L.rows && off < last && !(bits >> (off & 31) & 1);
                load_if(x[u], kc + off * m.token_stride + L.a, in[u]);
                load_if(y[u], kc + off * m.token_stride + L.b, in[u] && L.b >= 0);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (in[u]) see(x[u], y[u]);
        }
    }
    for (int r = 1; r < L.rows; ++r) {  // the lanes of the first row take the others'
        const int from = (lane + r * L.per_row) & 31;
        auto other = [&](const Piece& x) {
            Piece y;
#pragma unroll
            for (int k = 0; k < V::kWords; ++k) word(y, k) = __shfl_sync(0xffffffffu, word(x, k), from);
            return y;
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const Piece l = other(lo[x]), h = other(hi[x]);
            if (lane < L.per_row) take<V, false>(lo[x], l), take<V, true>(hi[x], h);
        }
    }
    if (split > 1) {
        red[sub][lane][0] = lo[0], red[sub][lane][1] = lo[1], red[sub][lane][2] = hi[0], red[sub][lane][3] = hi[1];
        __syncthreads();
        for (int w = 1; w < split; ++w)
#pragma unroll
            for (int x = 0; x < 2; ++x) take<V, false>(lo[x], red[w][lane][x]), take<V, true>(hi[x], red[w][lane][2 + x]);
        __syncthreads();
    }
    if (sub == 0 && lane < L.per_row) {
        T* dst = (T*)a.k_bounds + ((int64_t)page * m.hkv + g) * 2 * m.d;
        *reinterpret_cast<Piece*>(dst + L.a) = lo[0];
        *reinterpret_cast<Piece*>(dst + m.d + L.a) = hi[0];
        if (L.b >= 0) {
            *reinterpret_cast<Piece*>(dst + L.b) = lo[1];
            *reinterpret_cast<Piece*>(dst + m.d + L.b) = hi[1];
        }
    }
}

// Blocks [0, check_blocks): what is wrong with the tokens, and the bounds of the pages whose first token of the call is
// among a unit's `slice`, at one kv head; a unit has `split` warps. The other blocks: rows.
template <typename V>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(PagedMeta m, AppendArgs a, int32_t* status, int64_t check_blocks,
                                                             int32_t slice, int32_t split) {
    __shared__ typename V::Piece red[kWarps][32][4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    after_previous();
    if (__syncthreads_or(status_bad(status))) return;
    if (blockIdx.x >= check_blocks) {
        append_rows<V>(m, a, (blockIdx.x - check_blocks) * kWarps + warp, lane, status);
        return;
    }
    const int32_t heads = a.k_bounds ? m.hkv : 1, sub = warp % split;
    const int64_t unit = ((int64_t)blockIdx.x * kWarps + warp) / split, i0 = unit / heads * slice;
    const int32_t g = (int32_t)(unit % heads);
    uint32_t firsts = page_firsts(m, a, i0, slice, lane, g == 0 && sub == 0, status);
    if (!a.k_bounds) return;
    for (; firsts; firsts &= firsts - 1) {
        const int64_t i = i0 + __ffs(firsts) - 1;
        const int32_t* row = a.table + a.token_seq[i] * m.table_stride;
        const int32_t page = paged_page(m, row, a.token_pos[i] >> m.page_shift, status);
        if (page >= 0) page_bounds<V>(m, a, i, page, g, split, sub, lane, red);
    }
}

template <typename V>
cudaError_t launch_pieces(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st) {
    using T = typename V::T;
    int sms = 0;
    const cudaError_t known = sm_count(&sms);
    if (known != cudaSuccess) return known;
    const int rows = 32 / (a.rope_dim / 2 / V::kN + ((m.d - a.rope_dim) / V::kN + 1) / 2);
    const int64_t units = (a.q ? Units(m.hq, 4 * rows).of(a.n_tokens) : 0) + Units(m.hkv, 2 * rows).of(a.n_tokens);
    const int64_t row_blocks = (units + kWarps - 1) / kWarps;
    // Tokens that are looked through for pages at a time: few where each may be a page of its own (1000 sequences' tokens,
    // 32/8 heads: 32 at a time 70 us, so 18), many where there are enough warps.
    const int32_t heads = a.k_bounds ? m.hkv : 1;
    const int32_t slice = (int32_t)std::min<int64_t>(32, std::max<int64_t>(1, a.n_tokens * heads / (sms * 16)));
    const int64_t slices = (a.n_tokens + slice - 1) / slice * heads;
    // One launch or two. 32/4 heads, d 128, bf16: 1 token 4.8 us and 5.1, 251 tokens, 32/8 heads (3012 warps' rows) 10.9 and
    // 11.6; 400 tokens of a sequence in pages of 64 (4000) 12.6 and 8.4, 16000 tokens 92 and 74.
    if (a.n_tokens * ((a.q ? m.hq : 0) + 2 * m.hkv) / rows < sms * 24) {
        // A page is shared by a block's warps where it is long (one token, pages of 128: 4.9 us, by one warp 6.0; of 1024: 12.5, 35.5).
        const int32_t split = a.k_bounds && m.page > 16 && slices <= sms * 8 ? kWarps : 1;
        const int64_t check_blocks = (slices * split + kWarps - 1) / kWarps;
        return note_error(launch_overlapped(append_kernel<V>, check_blocks + row_blocks, kThreads, 0, st, m, a, status,
                                            check_blocks, slice, split),
                          "paged append");
    }
    cudaError_t e = launch_overlapped(append_rows_kernel<V>, row_blocks, kThreads, 0, st, m, a, status);
    if (e == cudaSuccess)
        e = launch_overlapped(append_bounds_kernel<T>, (slices + kWarps - 1) / kWarps, kThreads, 0, st, m, a, status, slice);
    return note_error(e, "paged append");
}

// 16 bytes a piece where half of rope_dim is a multiple of them, 8 where it is of those (16000 tokens, 32/4 heads, d 80,
// rope_dim 40 in bf16: 65 us; rope_dim 80, 16 bytes: 54; rope_dim 20, channel by channel: 188), else channel by channel.
template <typename T>
cudaError_t launch(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st) {
    const int half = a.rope_dim / 2;
    if (half % Vec<T, uint4>::kN == 0) return launch_pieces<Vec<T, uint4>>(m, a, status, st);
    if (half % Vec<T, uint2>::kN == 0) return launch_pieces<Vec<T, uint2>>(m, a, status, st);
    append_channels_kernel<T><<<(unsigned)a.n_tokens, 128, 0, st>>>(m, a, status);
    if (a.k_bounds) append_channels_bounds_kernel<T><<<(unsigned)a.n_tokens, 128, 0, st>>>(m, a, status);
    return note_error(cudaGetLastError(), "paged append");
}

}  // namespace

cudaError_t launch_paged_append(const PagedMeta& m, const AppendArgs& a, int32_t* status, cudaStream_t st) {
    return m.dtype == SPLITKV_BF16 ? launch<__nv_bfloat16>(m, a, status, st) : launch<float>(m, a, status, st);
}

}  // namespace splitkv
