// Attention of one new token of each sequence over a paged key-value cache, split over the cache's length and joined.
//
// One pass with a running maximum and sum: for a tile of 16 keys, S^T = K Q^T (m16n8k16: 16 keys x 8 query rows of a kv
// head), P = exp2(S - m), O^T += V^T P^T. Keys are the M rows, so a group of 8 query heads fills the instruction (with
// queries as M, half of it or more would be padding), and both operands come straight from global memory: the order
// of the channels inside a dot product and of the output's channels over the lanes is free, so a lane's 16-byte load
// of a K row holds its fragments of two k-steps, and pairs of V rows become fragments by byte permutes. Nothing goes
// through shared memory on the way in. The work is bound by the bytes of K and V (one multiply-add per 2 bytes).
//
// All (sequence, kv head, tile) units form one line that is cut into equal parts, a part per block and again per
// warp, so that ragged batches load every SM alike. What a warp finishes alone it writes out; parts of a segment
// (sequence, kv head, group of query rows) are joined by their log-sum-exp, first in shared memory, then, for segments
// that several blocks hold, by the last of them to arrive, in the order of the blocks (results do not depend on which
// one is last).
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "sm100.cuh"

namespace splitkv {
namespace {

using sm100::ex2_approx;

constexpr int kTile = 16;          // keys of a unit
constexpr int kMaxParts = 512;     // most blocks that share the work: counters and partial slots of the workspace
constexpr size_t kCounterBytes = 4096;
constexpr float kLazy = 8.f;       // log2 units a score may exceed the reference before the reference moves
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxDP = 128, kMaxRows = 16;

static_assert(kMaxParts * sizeof(uint32_t) <= kCounterBytes, "counters");

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// D += A B for one 16x8 tile, bf16 x bf16 -> f32 (16 deep) or tf32 x tf32 -> f32 (8 deep).
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t to_tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// x = hi + lo with both in tf32, up to 2^-21 |x|. hi is cut, not rounded, so that it stays finite.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = to_tf32(x - __uint_as_float(hi));
}

// The 16 cache rows of a tile, one per lane (lanes 16.. repeat 0..): element offset at the kv head, or not to be read.
struct TileRows {
    int64_t off;
    uint32_t valid;  // bit r: row r is read
};

// ---- fragments of one warp: NT tiles of 8 query rows, DP channels (d rounded up to 64 or 128; the rest is zero)
template <typename T, int DP, int NT>
struct Frag;

template <int DP, int NT>
struct Frag<__nv_bfloat16, DP, NT> {
    using T = __nv_bfloat16;
    static constexpr int kOut = DP / 16;  // 16-channel tiles of the output
    uint4 q[NT][DP / 32];
    uint4 k[DP / 32][2];
    uint4 v[DP / 64][4];
    float o[NT][kOut][4];

    // Query rows of the group: `rows` of them from `base`; lane (g, t) holds row g's channels 32j + 8t ..
    __device__ __forceinline__ void load_q(const T* base, int rows, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) {
                const int c = 32 * j + 8 * t;
                q[n][j] = n * 8 + g < rows && c < d
                              ? __ldg(reinterpret_cast<const uint4*>(base + (int64_t)(n * 8 + g) * d + c))
                              : make_uint4(0, 0, 0, 0);
            }
    }
    __device__ __forceinline__ void load_k(const T* kc, const TileRows& r, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t off = __shfl_sync(0xffffffffu, r.off, g + 8 * x);
            const bool in = r.valid >> (g + 8 * x) & 1;
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) {
                const int c = 32 * j + 8 * t;
                k[j][x] = in && c < d ? ldg_stream(kc + off + c) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void load_v(const T* vc, const TileRows& r, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int key = 2 * t + (x & 1) + 8 * (x >> 1);
            const int64_t off = __shfl_sync(0xffffffffu, r.off, key);
            const bool in = r.valid >> key & 1;
#pragma unroll
            for (int c0 = 0; c0 < DP / 64; ++c0) {
                const int c = 64 * c0 + 8 * g;
                v[c0][x] = in && c < d ? ldg_stream(vc + off + c) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    // s[n]: keys g, g + 8 (s[0..1], s[2..3]) x query rows 2t, 2t + 1.
    __device__ __forceinline__ void scores(float (&s)[NT][4]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float a[2][4] = {};  // two chains: the instructions of one depend on each other
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) {
                mma_bf16(a[0], k[j][0].x, k[j][1].x, k[j][0].y, k[j][1].y, q[n][j].x, q[n][j].y);
                mma_bf16(a[1], k[j][0].z, k[j][1].z, k[j][0].w, k[j][1].w, q[n][j].z, q[n][j].w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = a[0][i] + a[1][i];
        }
    }
    // O += P V. P goes in as two bf16 halves (2^-17 together): with one, its rounding would add as much error to the
    // output as the output's own rounding; the second product costs nothing, the loads bound the kernel.
    __device__ __forceinline__ void values(const float (&p)[NT][4], int lane) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t hi = pack_bf16(p[n][2 * x], p[n][2 * x + 1]);
                const float r0 = p[n][2 * x] - __uint_as_float(hi << 16);
                const float r1 = p[n][2 * x + 1] - __uint_as_float(hi & 0xffff0000u);
                b[n][x] = transpose8x8(hi);
                b[n][2 + x] = transpose8x8(pack_bf16(r0, r1));
            }
#pragma unroll
        for (int c0 = 0; c0 < DP / 64; ++c0) {
            const uint32_t* r[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) r[x] = reinterpret_cast<const uint32_t*>(&v[c0][x]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t a0 = __byte_perm(r[0][w], r[1][w], 0x5410), a1 = __byte_perm(r[0][w], r[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(r[2][w], r[3][w], 0x5410), a3 = __byte_perm(r[2][w], r[3][w], 0x7632);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(o[n][4 * c0 + w], a0, a1, a2, a3, b[n][0], b[n][1]);
                    mma_bf16(o[n][4 * c0 + w], a0, a1, a2, a3, b[n][2], b[n][3]);
                }
            }
        }
    }
    // The lane's channels of query row n*8 + 2t + y: fn(first channel, 4 values).
    template <typename F>
    __device__ __forceinline__ void each(int n, int y, int lane, F&& fn) const {
#pragma unroll
        for (int c0 = 0; c0 < DP / 64; ++c0)
#pragma unroll
            for (int w = 0; w < 4; w += 2) {
                const auto &x = o[n][4 * c0 + w], &z = o[n][4 * c0 + w + 1];
                fn(64 * c0 + 8 * (lane >> 2) + 2 * w, make_float4(x[y], x[2 + y], z[y], z[2 + y]));
            }
    }
};

// float32: each product as three tf32 products of the operands' halves (what is left out is below 2^-21 of it).
template <int DP, int NT>
struct Frag<float, DP, NT> {
    using T = float;
    static constexpr int kOut = DP / 16;
    float4 q[NT][DP / 16];
    float4 k[DP / 16][2];
    float4 v[DP / 32][4];
    float o[NT][kOut][4];

    static __device__ __forceinline__ float4 load(const T* p) {
        const uint4 r = ldg_stream(p);
        return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ __forceinline__ void load_q(const T* base, int rows, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                const int c = 16 * j + 4 * t;
                q[n][j] = n * 8 + g < rows && c < d
                              ? __ldg(reinterpret_cast<const float4*>(base + (int64_t)(n * 8 + g) * d + c))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            }
    }
    __device__ __forceinline__ void load_k(const T* kc, const TileRows& r, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t off = __shfl_sync(0xffffffffu, r.off, g + 8 * x);
            const bool in = r.valid >> (g + 8 * x) & 1;
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                const int c = 16 * j + 4 * t;
                k[j][x] = in && c < d ? load(kc + off + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
    __device__ __forceinline__ void load_v(const T* vc, const TileRows& r, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t off = __shfl_sync(0xffffffffu, r.off, t + 4 * x);
            const bool in = r.valid >> (t + 4 * x) & 1;
#pragma unroll
            for (int c0 = 0; c0 < DP / 32; ++c0) {
                const int c = 32 * c0 + 4 * g;
                v[c0][x] = in && c < d ? load(vc + off + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
    // acc += a b over 8 channels, a [16 x 8] as four values a lane. An infinite value has no halves: kInf keeps it to
    // the product of the high ones.
    template <bool kInf = false>
    static __device__ __forceinline__ void product(float (&acc)[NT][4], const float (&a)[4], const float (&b0)[NT],
                                                   const float (&b1)[NT]) {
        uint32_t hi[4], lo[4], fin[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            split_tf32(a[i], hi[i], lo[i]);
            fin[i] = hi[i];
            if (kInf && !isfinite(a[i])) lo[i] = fin[i] = 0;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t h0, l0, h1, l1;
            split_tf32(b0[n], h0, l0);
            split_tf32(b1[n], h1, l1);
            uint32_t f0 = h0, f1 = h1;
            if (kInf && !isfinite(b0[n])) l0 = f0 = 0;
            if (kInf && !isfinite(b1[n])) l1 = f1 = 0;
            mma_tf32(acc[n], lo, f0, f1);
            mma_tf32(acc[n], fin, l0, l1);
            mma_tf32(acc[n], hi, h0, h1);
        }
    }
    __device__ __forceinline__ void scores(float (&s)[NT][4]) const {
        sums<false>(s);
        bool nan = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= s[n][i] != s[n][i];
        if (__any_sync(0xffffffffu, nan)) sums<true>(s);  // infinite keys or queries
    }
    template <bool kInf>
    __device__ __forceinline__ void sums(float (&s)[NT][4]) const {
        float a[2][NT][4] = {};
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
            float b0[NT], b1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b0[n] = q[n][j].x, b1[n] = q[n][j].y;
            product<kInf>(a[0], {k[j][0].x, k[j][1].x, k[j][0].y, k[j][1].y}, b0, b1);
#pragma unroll
            for (int n = 0; n < NT; ++n) b0[n] = q[n][j].z, b1[n] = q[n][j].w;
            product<kInf>(a[1], {k[j][0].z, k[j][1].z, k[j][0].w, k[j][1].w}, b0, b1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = a[0][n][i] + a[1][n][i];
    }
    __device__ __forceinline__ void values(const float (&p)[NT][4], int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // keys 8x .. 8x + 7
            float b0[NT], b1[NT];      // P at (key 8x + t, row g) and (key 8x + t + 4, row g)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float e0 = __shfl_sync(0xffffffffu, p[n][2 * x], t * 4 + (g >> 1));
                const float e1 = __shfl_sync(0xffffffffu, p[n][2 * x + 1], t * 4 + (g >> 1));
                const float f0 = __shfl_sync(0xffffffffu, p[n][2 * x], (t + 4) * 4 + (g >> 1));
                const float f1 = __shfl_sync(0xffffffffu, p[n][2 * x + 1], (t + 4) * 4 + (g >> 1));
                b0[n] = g & 1 ? e1 : e0;
                b1[n] = g & 1 ? f1 : f0;
            }
#pragma unroll
            for (int c0 = 0; c0 < DP / 32; ++c0) {
                const float4 &y = v[c0][2 * x], &z = v[c0][2 * x + 1];
                float acc[NT][4];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] = o[n][2 * c0 + w][i];
                    if (w == 0)
                        product(acc, {y.x, y.y, z.x, z.y}, b0, b1);
                    else
                        product(acc, {y.z, y.w, z.z, z.w}, b0, b1);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[n][2 * c0 + w][i] = acc[n][i];
                }
            }
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(int n, int y, int lane, F&& fn) const {
#pragma unroll
        for (int c0 = 0; c0 < DP / 32; ++c0) {
            const auto &x = o[n][2 * c0], &z = o[n][2 * c0 + 1];
            fn(32 * c0 + 4 * (lane >> 2), make_float4(x[y], x[2 + y], z[y], z[2 + y]));
        }
    }
};

__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

// Everything a block needs to know about the line of units.
struct Line {
    const int32_t* prefix;  // shared: tiles of the sequences before b (of one kv head)
    int32_t n_seqs, per_seq;  // per_seq = kv heads x groups of query rows: segments of a sequence
    int64_t total;
    int32_t parts;

    __device__ __forceinline__ int64_t lo(int64_t c) const { return total * c / parts; }
    __device__ __forceinline__ int32_t part_of(int64_t u) const {  // the part that holds unit u
        return (int32_t)(((u + 1) * parts - 1) / total);
    }
};

// One segment as seen from a unit of it.
struct Segment {
    int32_t b, sub, tile, tiles;  // sequence, kv head and row group, tile of the unit, tiles in all
    int64_t start;                // first unit
};

__device__ __forceinline__ Segment segment_at(const Line& L, int64_t u) {
    int32_t lo = 0, hi = L.n_seqs;  // the last b with prefix[b] * per_seq <= u
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if ((int64_t)L.prefix[mid] * L.per_seq <= u) lo = mid; else hi = mid;
    }
    Segment s;
    s.b = lo;
    s.tiles = L.prefix[lo + 1] - L.prefix[lo];
    const int64_t rem = u - (int64_t)L.prefix[lo] * L.per_seq;
    s.sub = (int32_t)(rem / s.tiles);
    s.tile = (int32_t)(rem - (int64_t)s.sub * s.tiles);
    s.start = u - s.tile;
    return s;
}

// A partial result: unnormalised O, reference maximum (log2 units) and sum of each row.
template <int DP, int R>
struct Partial {
    float o[R][DP];
    float m[R], l[R];
};

template <typename T, int DP, int NT, int W>
__global__ void __launch_bounds__(W * 32, 1) decode_kernel(PagedMeta m, const T* __restrict__ q, int64_t q_stride,
                                                          const T* __restrict__ kc, const T* __restrict__ vc,
                                                          const int32_t* __restrict__ table,
                                                          const int32_t* __restrict__ seq_len,
                                                          const int32_t* __restrict__ pages, int32_t n_select,
                                                          T* __restrict__ o, float* __restrict__ lse, int32_t* status,
                                                          uint32_t* counters, char* slots) {
    constexpr int R = 8 * NT;
    using P = Partial<DP, R>;
    extern __shared__ __align__(16) char smem[];
    P* part = reinterpret_cast<P*>(smem);  // [W][2]
    __shared__ int64_t seg_of[W][2];       // first unit of the segment a warp's partial belongs to, -1: none
    __shared__ int32_t shared_flag[3];     // status seen, and whether this block joins its left, its right segment
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + sizeof(P) * W * 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row_groups = (m.group + R - 1) / R;

    // ---- the line of units
    if (tid == 0) shared_flag[0] = status_bad(status);
    for (int b = tid; b < m.n_seqs; b += W * 32) {
        const int32_t len = paged_len(m, seq_len, b, status);
        int32_t n = len;
        if (pages) n = min(n_select, (len + m.page - 1) >> m.page_shift) << m.page_shift;
        prefix[b + 1] = (n + kTile - 1) / kTile;
    }
    __syncthreads();
    if (warp == 0) {
        int32_t carry = 0;
        for (int b0 = 0; b0 < m.n_seqs; b0 += 32) {
            int32_t x = b0 + lane < m.n_seqs ? prefix[b0 + lane + 1] : 0;
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
    const bool skip = shared_flag[0];
    Line L{prefix, m.n_seqs, m.hkv * row_groups, 0, 0};
    L.total = (int64_t)prefix[m.n_seqs] * L.per_seq;
    const int64_t want = (L.total + W - 1) / W;
    L.parts = (int32_t)(want < gridDim.x ? want : gridDim.x);

    // ---- sequences without keys
    if (!skip)
        for (int b = blockIdx.x; b < m.n_seqs; b += gridDim.x) {
            if (prefix[b + 1] > prefix[b]) continue;
            for (int i = tid; i < m.hq * m.d; i += W * 32) o[(int64_t)b * m.hq * m.d + i] = from_f32<T>(0.f);
            for (int h = tid; h < m.hq; h += W * 32) lse[(int64_t)b * m.hq + h] = -INFINITY;
            if (pages)
                for (int i = tid; i < m.hkv * n_select; i += W * 32)
                    if (pages[(int64_t)b * m.hkv * n_select + i] != -1) raise_status(status, SPLITKV_DEV_BAD_PAGE);
        }
    if ((int)blockIdx.x >= L.parts) return;

    const int64_t c_lo = L.lo(blockIdx.x), c_hi = L.lo(blockIdx.x + 1);
    const int64_t w_lo = c_lo + (c_hi - c_lo) * warp / W, w_hi = c_lo + (c_hi - c_lo) * (warp + 1) / W;
    if (lane < 2) seg_of[warp][lane] = -1;
    __syncwarp();

    Frag<T, DP, NT> f;
    const float to_log2 = m.scale * kLog2e;
    for (int64_t u = skip ? w_hi : w_lo; u < w_hi;) {
        const Segment sg = segment_at(L, u);
        const int32_t t_end = (int32_t)(w_hi - sg.start < sg.tiles ? w_hi - sg.start : sg.tiles);
        const int32_t g = sg.sub / row_groups, row0 = (sg.sub - g * row_groups) * R;
        const int32_t rows = min(R, m.group - row0);
        const int32_t* trow = table + sg.b * m.table_stride;
        const int32_t len = __ldg(seq_len + sg.b), count = (len + m.page - 1) >> m.page_shift;
        const int32_t* list = pages ? pages + ((int64_t)sg.b * m.hkv + g) * n_select : nullptr;
        const int32_t listed = list ? min(n_select, count) : 0;
        const int64_t head = (int64_t)g * m.head_stride;
        f.load_q(q + sg.b * q_stride + (int64_t)(g * m.group + row0) * m.d, rows, m.d, lane);
        if (list && sg.tile == 0 && row0 == 0)  // the unread tail of the list has to be empty
            for (int32_t i = listed + lane; i < n_select; i += 32)
                if (__ldg(list + i) != -1) raise_status(status, SPLITKV_DEV_BAD_PAGE);

        // Page-table entry of the lane's row of tile i, or -1 (past the end, or not listed).
        auto entry_of = [&](int32_t i) -> int32_t {
            const int32_t pos = i * kTile + (lane & 15), e = pos >> m.page_shift;
            if (i >= t_end) return -1;
            if (!list) return pos < len ? e : -1;
            if (e >= listed) return -1;
            const int32_t x = __ldg(list + e);
            const bool first = (pos & (m.page - 1)) == 0 || (lane & 15) == 0;
            if (x < -1 || x >= count) {
                raise_status(status, SPLITKV_DEV_BAD_PAGE);
                return -1;
            }
            if (first && e > 0 && x >= 0) {
                const int32_t y = __ldg(list + e - 1);
                if (y < 0 || y >= x) raise_status(status, SPLITKV_DEV_BAD_PAGE);
            }
            return x;
        };
        auto page_of = [&](int32_t e) -> int32_t { return e < 0 ? -1 : paged_page(m, trow, e, status); };
        auto rows_of = [&](int32_t i, int32_t e, int32_t page) -> TileRows {
            const int32_t off = (i * kTile + (lane & 15)) & (m.page - 1);
            TileRows r;
            const bool in = page >= 0 && (e << m.page_shift) + off < len;
            r.off = in ? page * m.page_stride + head + off * m.token_stride : 0;
            r.valid = __ballot_sync(0xffffffffu, in) & 0xffffu;
            return r;
        };

        float mx[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int y = 0; y < 2; ++y) mx[n][y] = -INFINITY, ref[n][y] = 0.f, l[n][y] = 0.f;
#pragma unroll
            for (int i = 0; i < Frag<T, DP, NT>::kOut; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f.o[n][i][j] = 0.f;
        }

        // Loads run ahead: K of the next tile is on its way during this one's softmax and PV, V during the next
        // one's QK; page-table entries two tiles ahead, list entries three.
        int32_t i = sg.tile;
        int32_t e0 = entry_of(i), e1 = entry_of(i + 1), e2 = entry_of(i + 2);
        int32_t p0 = page_of(e0), p1 = page_of(e1);
        TileRows r = rows_of(i, e0, p0);
        f.load_k(kc, r, m.d, lane);
        f.load_v(vc, r, m.d, lane);
        for (; i < t_end; ++i) {
            const uint32_t valid = r.valid;
            r = rows_of(i + 1, e1, p1);
            e1 = e2;
            p1 = page_of(e1);
            e2 = entry_of(i + 3);
            float s[NT][4];
            f.scores(s);
            f.load_k(kc, r, m.d, lane);
            const bool in0 = valid >> (lane >> 2) & 1, in1 = valid >> ((lane >> 2) + 8) & 1;
            bool move = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    s[n][y] = in0 ? s[n][y] * to_log2 : -INFINITY;
                    s[n][2 + y] = in1 ? s[n][2 + y] * to_log2 : -INFINITY;
                    move |= fmaxf(s[n][y], s[n][2 + y]) > mx[n][y] + kLazy;
                }
            }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = fmaxf(s[n][y], s[n][2 + y]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        if (top > mx[n][y]) {
                            const float fix = ex2_approx(mx[n][y] - top);  // 0 from the start's -inf
                            mx[n][y] = ref[n][y] = top;
                            l[n][y] *= fix;
#pragma unroll
                            for (int j = 0; j < Frag<T, DP, NT>::kOut; ++j)
                                f.o[n][j][y] *= fix, f.o[n][j][2 + y] *= fix;
                        }
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    s[n][y] = ex2_approx(s[n][y] - ref[n][y]);
                    s[n][2 + y] = ex2_approx(s[n][2 + y] - ref[n][y]);
                    l[n][y] += s[n][y] + s[n][2 + y];
                }
            f.values(s, lane);
            f.load_v(vc, r, m.d, lane);
        }

        // The rows' sums over the lanes that hold their keys.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][y] += __shfl_xor_sync(0xffffffffu, l[n][y], x);
        const int t = lane & 3;
        if (sg.tile == 0 && t_end == sg.tiles) {  // a whole segment
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = 8 * n + 2 * t + y;
                    if (row >= rows) continue;
                    const int64_t h = (int64_t)sg.b * m.hq + g * m.group + row0 + row;
                    const float inv = l[n][y] == 0.f ? 0.f : 1.f / l[n][y];
                    f.each(n, y, lane, [&](int c, float4 x) {
                        if (c < m.d) store4(o + h * m.d + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                    });
                    if (lane < 4) lse[h] = l[n][y] == 0.f ? -INFINITY : (mx[n][y] + log2f(l[n][y])) * (1.f / kLog2e);
                }
        } else {
            const int slot = seg_of[warp][0] >= 0;
            __syncwarp();
            P& out = part[warp * 2 + slot];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = 8 * n + 2 * t + y;
                    f.each(n, y, lane, [&](int c, float4 x) { *reinterpret_cast<float4*>(&out.o[row][c]) = x; });
                    if (lane < 4) out.m[row] = mx[n][y], out.l[row] = l[n][y];
                }
            if (lane == 0) seg_of[warp][slot] = sg.start;
            __syncwarp();
        }
        u = sg.start + t_end;
    }
    __syncthreads();

    // ---- join the warps' parts, segment by segment
    P* const mine = reinterpret_cast<P*>(slots) + blockIdx.x * 2;
    auto finish = [&](const Segment& sg, int row, int c, float4 acc, float mm, float ll) {
        const int32_t g = sg.sub / row_groups, r0 = (sg.sub - g * row_groups) * R;
        if (r0 + row >= m.group || c >= m.d) return;
        const int64_t h = (int64_t)sg.b * m.hq + g * m.group + r0 + row;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        store4(o + h * m.d + c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (c == 0) lse[h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * (1.f / kLog2e);
    };
    if (!skip) {
        for (int i = 0; i < 2 * W;) {
            const int64_t start = seg_of[i >> 1][i & 1];
            if (start < 0) {
                ++i;
                continue;
            }
            int n = i + 1;
            while (n < 2 * W && (seg_of[n >> 1][n & 1] == start || seg_of[n >> 1][n & 1] < 0)) ++n;
            const Segment sg = segment_at(L, start);
            const bool whole = start >= c_lo && start + sg.tiles <= c_hi;
            for (int x = tid; x < R * DP / 4; x += W * 32) {
                const int row = x / (DP / 4), c = x % (DP / 4) * 4;
                float mm = -INFINITY, ll = 0.f;
                for (int k = i; k < n; ++k)
                    if (seg_of[k >> 1][k & 1] >= 0) mm = fmaxf(mm, part[k].m[row]);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = i; k < n; ++k) {
                    if (seg_of[k >> 1][k & 1] < 0 || part[k].m[row] == -INFINITY) continue;
                    const float w = ex2_approx(part[k].m[row] - mm);
                    const float4 y = *reinterpret_cast<const float4*>(&part[k].o[row][c]);
                    acc.x += w * y.x, acc.y += w * y.y, acc.z += w * y.z, acc.w += w * y.w;
                    ll += w * part[k].l[row];
                }
                if (whole) {
                    finish(sg, row, c, acc, mm, ll);
                } else {
                    P& out = mine[start >= c_lo];
                    *reinterpret_cast<float4*>(&out.o[row][c]) = acc;
                    if (c == 0) out.m[row] = mm, out.l[row] = ll;
                }
            }
            i = n;
        }
    }

    // ---- join the blocks' parts: side 0 is the segment that began in an earlier block, side 1 the one that goes on
    Segment side[2];
    bool open[2];
    side[0] = segment_at(L, c_lo);
    open[0] = side[0].start < c_lo;
    side[1] = segment_at(L, c_hi - 1);
    open[1] = side[1].start >= c_lo && side[1].start + side[1].tiles > c_hi;
    if (!open[0] && !open[1]) return;
    __threadfence();
    __syncthreads();
    if (tid < 2) {
        int32_t last = 0;
        if (open[tid]) {
            const int32_t first = L.part_of(side[tid].start), end = L.part_of(side[tid].start + side[tid].tiles - 1);
            // Counts up to the number of blocks and wraps to 0 by itself: ready for the next call. A block that
            // skipped its work for the status word's sake arrives all the same.
            last = atomicInc(counters + first, end - first) == (uint32_t)(end - first);
            __threadfence();
        }
        shared_flag[1 + tid] = last;
    }
    __syncthreads();
    if (skip) return;
    for (int s = 0; s < 2; ++s) {
        if (!open[s] || !shared_flag[1 + s]) continue;
        const int32_t first = L.part_of(side[s].start), end = L.part_of(side[s].start + side[s].tiles - 1);
        const P* all = reinterpret_cast<const P*>(slots);
        for (int x = tid; x < R * DP / 4; x += W * 32) {
            const int row = x / (DP / 4), c = x % (DP / 4) * 4;
            float mm = -INFINITY, ll = 0.f;
            for (int k = first; k <= end; ++k) mm = fmaxf(mm, __ldcg(&all[2 * k + (k == first)].m[row]));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = first; k <= end; ++k) {
                const P& y = all[2 * k + (k == first)];
                const float pm = __ldcg(&y.m[row]), pl = __ldcg(&y.l[row]);
                const float4 z = __ldcg(reinterpret_cast<const float4*>(&y.o[row][c]));
                const float w = pm == -INFINITY ? 0.f : ex2_approx(pm - mm);
                acc.x += w * z.x, acc.y += w * z.y, acc.z += w * z.z, acc.w += w * z.w;
                ll += w * pl;
            }
            finish(side[s], row, c, acc, mm, ll);
        }
    }
}

template <typename T, int DP, int NT, int W>
cudaError_t launch(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                   const int32_t* table, const int32_t* seq_len, const int32_t* pages, int32_t n_select, void* o,
                   float* lse, int32_t* status, void* ws, cudaStream_t st) {
    using P = Partial<DP, 8 * NT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return note_error(e, "paged decode: device");
    const size_t smem = sizeof(P) * W * 2 + sizeof(int32_t) * (m.n_seqs + 1);
    auto kern = decode_kernel<T, DP, NT, W>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return note_error(e, "paged decode: shared memory");
    const int grid = std::min(sms, kMaxParts);
    kern<<<grid, W * 32, smem, st>>>(m, (const T*)q, q_stride, (const T*)k_cache, (const T*)v_cache, table, seq_len,
                                     pages, n_select, (T*)o, lse, status, (uint32_t*)ws, (char*)ws + kCounterBytes);
    return note_error(cudaGetLastError(), "paged decode");
}

}  // namespace

size_t paged_decode_workspace(const PagedMeta&) {
    return kCounterBytes + sizeof(Partial<kMaxDP, kMaxRows>) * kMaxParts * 2;
}

cudaError_t launch_paged_decode(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, const int32_t* table, const int32_t* seq_len,
                                const int32_t* pages, int32_t n_select, void* o, float* lse, int32_t* status, void* ws,
                                cudaStream_t st) {
#define SPLITKV_DECODE(T, DP, NT, W) \
    launch<T, DP, NT, W>(m, q, q_stride, k_cache, v_cache, table, seq_len, pages, n_select, o, lse, status, ws, st)
    if (m.dtype == SPLITKV_F32) return m.d <= 64 ? SPLITKV_DECODE(float, 64, 1, 12) : SPLITKV_DECODE(float, 128, 1, 8);
    if (m.group > 8)
        return m.d <= 64 ? SPLITKV_DECODE(__nv_bfloat16, 64, 2, 12) : SPLITKV_DECODE(__nv_bfloat16, 128, 2, 8);
    return m.d <= 64 ? SPLITKV_DECODE(__nv_bfloat16, 64, 1, 16) : SPLITKV_DECODE(__nv_bfloat16, 128, 1, 12);
#undef SPLITKV_DECODE
}

}  // namespace splitkv
