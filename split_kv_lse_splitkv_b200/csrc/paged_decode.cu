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
constexpr int kMaxParts = 192;     // most blocks that share the work: counters and partial slots of the workspace
constexpr size_t kCounterBytes = 1024;
// Units that the beginning of a segment counts. 64 sequences of 1 .. 16384 keys, 8 kv heads: 0 units 168 us, 2: 98, 4: 84,
// 8: 85, 16: 86 (with 0 the short ones pile up on a few warps).
constexpr int kSegmentCost = 4;
// Most units of a segment that a block takes whole, without a join of blocks. One sequence, 4 kv heads, 8 warps: 333 keys
// (25 units) 10.2 us so and 11.4 us split, 440 keys 11.1 and 11.4, 500 keys (36 units) 11.6 and 11.2; d 64, 12 warps: 440
// keys 9.2 and 10.2, 500 keys 9.6 and 10.4. float32, d 64: 320 keys (24 units) 11.8 both, 380 keys 13.1 and 12.1.
template <typename T, int W>
constexpr int kAlone = sizeof(T) == 4 ? 24 : W > 10 ? 36 : 32;
constexpr float kLazy = 8.f;       // log2 units a score may exceed the reference before the reference moves
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kNone = ~0u;

static_assert(kMaxParts * sizeof(uint32_t) <= kCounterBytes, "counters");

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
// x = hi + lo with both in tf32, up to 2^-22 |x|. kCut: hi is cut, not rounded, so that it is finite where x is (up to
// 2^-21 |x| then).
template <bool kCut>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = kCut ? __float_as_uint(x) & 0xffffe000u : to_tf32(x);
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
    static constexpr int kShared = 0;
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
                              ? *reinterpret_cast<const uint4*>(base + (int64_t)(n * 8 + g) * d + c)
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
                k[j][x] = ldg_stream_if(kc + off + c, in && c < d);
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
                v[c0][x] = ldg_stream_if(vc + off + c, in && c < d);
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
    // output as the output's own rounding; the second product costs nothing, the loads bound the kernel. O adds up in the
    // tensor core, which cuts what its float32 sums do not hold. Products formed apart and added here, as in float32 below,
    // would change 0.13% of the outputs of 131071 keys by their last bit (0.36% differ from the rounded exact ones, 0.23%
    // then), none at 32768 keys, and take longer (32768 keys 22.7 us, 24.6 so; 256 x 100 keys 36.5, 41).
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
    static constexpr int kShared = NT * DP / 16;  // 16-byte pieces a lane keeps in shared memory: its queries
    float4* q;                                    // [NT][DP / 16][32]: they would not fit the registers beside K, V and O
    float4 k[DP / 16][2];
    float4 v[DP / 32][4];
    float o[NT][kOut][4];

    static __device__ __forceinline__ float4 load(const T* p, bool in) {
        const uint4 r = ldg_stream_if(p, in);
        return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ __forceinline__ void load_q(const T* base, int rows, int d, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
                const int c = 16 * j + 4 * t;
                q[(n * DP / 16 + j) * 32 + lane] =
                    n * 8 + g < rows && c < d
                        ? *reinterpret_cast<const float4*>(base + (int64_t)(n * 8 + g) * d + c)
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
                k[j][x] = load(kc + off + c, in && c < d);
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
                v[c0][x] = load(vc + off + c, in && c < d);
            }
        }
    }
    // acc += a b over 8 channels, a [16 x 8] as four values a lane. Formed apart and added in float32: the tensor core cuts
    // what its sums do not hold, always toward zero, and over a long row that would add up (1.3e-6 of o over 10^4 keys;
    // 3e-7 so). kCut: a may be as large as the type goes. kInf: a or b may be infinite and have no halves then; only the
    // product of the high ones sees it.
    template <bool kCut, bool kInf>
    static __device__ __forceinline__ void product(float (&acc)[NT][4], const float (&a)[4], const float (&b0)[NT],
                                                   const float (&b1)[NT]) {
        uint32_t hi[4], lo[4], fin[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            split_tf32<kCut>(a[i], hi[i], lo[i]);
            fin[i] = hi[i];
            if (kInf && !isfinite(a[i])) lo[i] = fin[i] = 0;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t h0, l0, h1, l1;
            split_tf32<kInf>(b0[n], h0, l0);
            split_tf32<kInf>(b1[n], h1, l1);
            uint32_t f0 = h0, f1 = h1;
            if (kInf && !isfinite(b0[n])) l0 = f0 = 0;
            if (kInf && !isfinite(b1[n])) l1 = f1 = 0;
            float d[4] = {};
            mma_tf32(d, lo, f0, f1);
            mma_tf32(d, fin, l0, l1);
            mma_tf32(d, hi, h0, h1);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += d[i];
        }
    }
    __device__ __forceinline__ void scores(float (&s)[NT][4]) const {
        sums<false>(s);
        bool nan = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= s[n][i] != s[n][i];
        if (__any_sync(0xffffffffu, nan)) sums<true>(s);  // infinite keys or queries, or near the type's end
    }
    template <bool kInf>
    __device__ __forceinline__ void sums(float (&s)[NT][4]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
            float b[4][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 y = q[(n * DP / 16 + j) * 32 + (threadIdx.x & 31)];
                b[0][n] = y.x, b[1][n] = y.y, b[2][n] = y.z, b[3][n] = y.w;
            }
            product<kInf, kInf>(s, {k[j][0].x, k[j][1].x, k[j][0].y, k[j][1].y}, b[0], b[1]);
            product<kInf, kInf>(s, {k[j][0].z, k[j][1].z, k[j][0].w, k[j][1].w}, b[2], b[3]);
        }
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
                float acc[2][NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[0][n][i] = o[n][2 * c0][i], acc[1][n][i] = o[n][2 * c0 + 1][i];
                product<true, false>(acc[0], {y.x, y.y, z.x, z.y}, b0, b1);
                product<true, false>(acc[1], {y.z, y.w, z.z, z.w}, b0, b1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][2 * c0][i] = acc[0][n][i], o[n][2 * c0 + 1][i] = acc[1][n][i];
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

// The line of units (fewer than 2^31: the launch sees to it). A segment (sequence, kv head, group of query rows)
// takes kSegmentCost units before its tiles': what it costs to begin one (table, queries, first keys: one after the
// other) next to the streaming of a tile.
struct Line {
    const uint32_t* prefix;    // shared: units of the sequences before b, for one segment of each
    uint32_t n_seqs, per_seq;  // per_seq = kv heads x groups of query rows: segments of a sequence
    uint32_t total, per_part;
};

struct Segment {
    int32_t b, sub, tiles;  // sequence, kv head and row group, tiles
    uint32_t start;         // first unit; its tiles begin at start + kSegmentCost
    __device__ __forceinline__ uint32_t tile0() const { return start + kSegmentCost; }
    __device__ __forceinline__ uint32_t end() const { return start + kSegmentCost + tiles; }
};

__device__ __forceinline__ Segment segment_at(const Line& L, uint32_t u) {
    uint32_t lo = 0;  // the last b with prefix[b] * per_seq <= u
    for (uint32_t hi = L.n_seqs; hi - lo > 1;) {
        const uint32_t mid = (lo + hi) >> 1;
        if (L.prefix[mid] * L.per_seq <= u) lo = mid; else hi = mid;
    }
    const uint32_t base = L.prefix[lo], width = L.prefix[lo + 1] - base;
    Segment s;
    s.b = lo;
    s.tiles = width - kSegmentCost;
    s.sub = (u - base * L.per_seq) / width;
    s.start = base * L.per_seq + s.sub * width;
    return s;
}

// A partial result: unnormalised O, reference maximum (log2 units) and sum of each row.
template <int DP, int R>
struct Partial {
    float o[R][DP];
    float m[R], l[R];
};

// A segment whose parts a block joins.
struct Group {
    int32_t first, n;  // its parts in the block's list of them
    int32_t rows;
    int32_t out;       // -1: the results; 0, 1: the block's part of the segment that it entered, that it leaves
    int64_t h;         // first row of the results
};

// A segment that several blocks hold.
struct Side {
    int32_t first, n;  // the blocks, 0: none
    int32_t rows, last;
    int64_t h;
};

template <typename T, int DP, int NT, int W>
__global__ void __launch_bounds__(W * 32, 1) decode_kernel(PagedMeta m, const T* q, int64_t q_stride, const T* kc,
                                                          const T* vc, const int32_t* table, const int32_t* seq_len,
                                                          const int32_t* pages, int32_t n_select, T* o, float* lse,
                                                          int32_t* status, uint32_t* counters, char* slots) {
    static_assert(2 * W <= 32, "one lane per partial of the block");
    constexpr int R = 8 * NT, kCols = DP / 4, kThreads = W * 32;
    using P = Partial<DP, R>;
    extern __shared__ __align__(16) char smem[];
    P* part = reinterpret_cast<P*>(smem);  // [W][2]: a warp's part of the segment it entered, of the one it left
    __shared__ uint32_t seg_of[2 * W];     // first unit of the segment that part belongs to, kNone: none
    __shared__ int32_t list[2 * W];        // the parts there are
    __shared__ float weight[2 * W][R];
    __shared__ float scale_of[2 * W][R];   // 1 / sum of a finished row
    __shared__ Group group[2 * W];
    __shared__ Side side[2];
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + sizeof(P) * W * 2 + Frag<T, DP, NT>::kShared * 512 * W);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row_groups = (m.group + R - 1) / R;

    after_previous();

    // ---- the line of units
    const bool bad = status_bad(status);
    auto units_of = [&](int b) {
        const int32_t len = paged_len(m, seq_len, b, status);
        int32_t n = len;
        if (pages) n = min(n_select, (len + m.page - 1) >> m.page_shift) << m.page_shift;
        return n ? (n + kTile - 1) / kTile + kSegmentCost : 0;
    };
    if (lane < 2) seg_of[warp * 2 + lane] = kNone;
    bool empties;      // some sequence has no keys
    int32_t widest;    // units of the longest segment
    if (m.n_seqs <= 32) {  // each warp by itself
        int32_t x = lane < m.n_seqs ? units_of(lane) : 0;
        empties = __any_sync(0xffffffffu, lane < m.n_seqs && x == 0);
        widest = __reduce_max_sync(0xffffffffu, x);
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
        int32_t most = 0;
        bool none = false;
        for (int b = tid; b < m.n_seqs; b += kThreads) {
            const int32_t x = units_of(b);
            prefix[b + 1] = x;
            none |= x == 0;
            most = max(most, x);
        }
        empties = __syncthreads_or(none);
        widest = __syncthreads_or(most > kAlone<T, W>) ? INT32_MAX : 0;
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
    const bool skip = __any_sync(0xffffffffu, bad);
    Line L{prefix, (uint32_t)m.n_seqs, (uint32_t)(m.hkv * row_groups), 0, 0};
    L.total = prefix[m.n_seqs] * L.per_seq;
    L.per_part = max((L.total - 1) / gridDim.x + 1, (uint32_t)W);

    // ---- sequences without keys
    if (empties && !skip)
        for (int b = blockIdx.x; b < m.n_seqs; b += gridDim.x) {
            if (prefix[b + 1] > prefix[b]) continue;
            for (int i = tid; i < m.hq * m.d; i += kThreads) o[(int64_t)b * m.hq * m.d + i] = from_f32<T>(0.f);
            for (int h = tid; h < m.hq; h += kThreads) lse[(int64_t)b * m.hq + h] = -INFINITY;
            if (pages)
                for (int i = tid; i < m.hkv * n_select; i += kThreads)
                    if (pages[(int64_t)b * m.hkv * n_select + i] != -1) raise_status(status, SPLITKV_DEV_BAD_PAGE);
        }
    // This block's part [c_lo, c_hi) of the line, and each warp's part of it.
    uint32_t c_lo = min(blockIdx.x * L.per_part, L.total), c_hi = min(c_lo + L.per_part, L.total);
    if (widest <= kAlone<T, W> && L.n_seqs * L.per_seq <= gridDim.x) {  // a block per segment
        const uint32_t b = blockIdx.x / L.per_seq;
        if (b >= L.n_seqs) return;
        const uint32_t width = prefix[b + 1] - prefix[b];
        c_lo = prefix[b] * L.per_seq + (blockIdx.x - b * L.per_seq) * width;
        c_hi = c_lo + width;
    }
    if (c_lo >= c_hi) return;
    const uint32_t each = (c_hi - c_lo) / W, more = (c_hi - c_lo) % W;
    const uint32_t w_lo = c_lo + warp * each + min((uint32_t)warp, more), w_hi = w_lo + each + ((uint32_t)warp < more);

    Frag<T, DP, NT> f;
    if constexpr (Frag<T, DP, NT>::kShared > 0)
        f.q = reinterpret_cast<float4*>(smem + sizeof(P) * W * 2) + warp * (Frag<T, DP, NT>::kShared * 32);
    const float to_log2 = m.scale * kLog2e;
    for (uint32_t u = skip ? w_hi : w_lo; u < w_hi;) {
        const Segment sg = segment_at(L, u);
        const int32_t t_begin = max((int32_t)(u - sg.tile0()), 0);
        u = min(w_hi, sg.end());
        const int32_t t_end = max((int32_t)(u - sg.tile0()), 0);
        if (t_end <= t_begin) continue;  // of this segment's units only those of its beginning
        const int32_t g = sg.sub / row_groups, row0 = (sg.sub - g * row_groups) * R;
        const int32_t rows = min(R, m.group - row0);
        const int32_t* trow = table + sg.b * m.table_stride;
        const int32_t len = seq_len[sg.b], count = (len + m.page - 1) >> m.page_shift;
        const int32_t* chosen = pages ? pages + ((int64_t)sg.b * m.hkv + g) * n_select : nullptr;
        const int32_t listed = chosen ? min(n_select, count) : 0;
        const int64_t head = (int64_t)g * m.head_stride;
        if (chosen && t_begin == 0 && row0 == 0)  // the unread tail of the list has to be empty
            for (int32_t i = listed + lane; i < n_select; i += 32)
                if (chosen[i] != -1) raise_status(status, SPLITKV_DEV_BAD_PAGE);

        // Page-table entry of the lane's row of tile i, or -1 (past the end, or not listed).
        auto entry_of = [&](int32_t i) -> int32_t {
            const int32_t pos = i * kTile + (lane & 15), e = pos >> m.page_shift;
            if (i >= t_end) return -1;
            if (!chosen) return pos < len ? e : -1;
            if (e >= listed) return -1;
            const int32_t x = chosen[e];
            const bool first = (pos & (m.page - 1)) == 0 || (lane & 15) == 0;
            if (x < -1 || x >= count) {
                raise_status(status, SPLITKV_DEV_BAD_PAGE);
                return -1;
            }
            if (first && e > 0 && x >= 0) {
                const int32_t y = chosen[e - 1];
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

        // Loads run ahead: K of the next tile is on its way during this one's softmax and PV, V during the next
        // one's QK; page-table entries two tiles ahead, list entries three.
        int32_t i = t_begin;
        int32_t e1 = entry_of(i + 1), e2 = entry_of(i + 2), p1;
        TileRows r;
        {
            const int32_t e0 = entry_of(i), p0 = page_of(e0);
            p1 = page_of(e1);
            f.load_q(q + sg.b * q_stride + (int64_t)(g * m.group + row0) * m.d, rows, m.d, lane);
            r = rows_of(i, e0, p0);
        }
        f.load_k(kc, r, m.d, lane);
        f.load_v(vc, r, m.d, lane);

        float mx[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int y = 0; y < 2; ++y) mx[n][y] = -INFINITY, ref[n][y] = 0.f, l[n][y] = 0.f;
#pragma unroll
            for (int x = 0; x < Frag<T, DP, NT>::kOut; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) f.o[n][x][j] = 0.f;
        }
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

        const int slot = warp * 2 + (t_begin == 0);
        const bool whole = t_begin == 0 && t_end == sg.tiles;
        const int64_t h0 = (int64_t)sg.b * m.hq + g * m.group + row0;
        P& out = part[slot];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = 8 * n + 2 * (lane & 3) + y;
                // The row's sum over the lanes that hold its keys.
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][y] += __shfl_xor_sync(0xffffffffu, l[n][y], x);
                if (!whole) {
                    f.each(n, y, lane, [&](int c, float4 x) { *reinterpret_cast<float4*>(&out.o[row][c]) = x; });
                    if (lane < 4) out.m[row] = mx[n][y], out.l[row] = l[n][y];
                } else if (row < rows) {
                    const float inv = l[n][y] == 0.f ? 0.f : 1.f / l[n][y];
                    f.each(n, y, lane, [&](int c, float4 x) {
                        if (c < m.d)
                            store4(o + (h0 + row) * m.d + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                    });
                    if (lane < 4)
                        lse[h0 + row] = l[n][y] == 0.f ? -INFINITY : (mx[n][y] + log2f(l[n][y])) * (1.f / kLog2e);
                }
            }
        if (!whole && lane == 0) seg_of[slot] = sg.start;
    }

    // ---- the segments that other blocks hold parts of: side 0 began in an earlier block, side 1 goes on in the next
    if (warp < 2) {
        const Segment sg = segment_at(L, warp ? c_hi - 1 : c_lo);
        const bool open = warp ? sg.tile0() >= c_lo && sg.tile0() < c_hi && sg.end() > c_hi : sg.tile0() < c_lo;
        if (lane == 0) {
            const int32_t g = sg.sub / row_groups, row0 = (sg.sub - g * row_groups) * R;
            Side x{0, 0, min(R, m.group - row0), 0, (int64_t)sg.b * m.hq + g * m.group + row0};
            if (open) {
                x.first = sg.tile0() / L.per_part;
                x.n = (sg.end() - 1) / L.per_part - x.first + 1;
            }
            side[warp] = x;
        }
    }
    __syncthreads();

    // ---- join the warps' parts
    P* const mine = reinterpret_cast<P*>(slots) + blockIdx.x * 2;
    int n_groups;
    {
        const uint32_t of = lane < 2 * W ? seg_of[lane] : kNone;
        const uint32_t valid = __ballot_sync(0xffffffffu, of != kNone), below = valid & ((1u << lane) - 1);
        const uint32_t before = __shfl_sync(0xffffffffu, of, below ? 31 - __clz(below) : 0);
        const uint32_t heads = __ballot_sync(0xffffffffu, of != kNone && (!below || before != of));
        n_groups = __popc(heads);
        if (warp == 0 && of != kNone) list[__popc(below)] = lane;
        for (int k = warp; k < n_groups; k += W) {
            uint32_t rest = heads;
            for (int i = 0; i < k; ++i) rest &= rest - 1;
            const int first = __ffs(rest) - 1;
            rest &= rest - 1;
            const uint32_t set = valid & ~((1u << first) - 1) & (rest ? (rest & -rest) - 1 : ~0u);
            const Segment sg = segment_at(L, __shfl_sync(0xffffffffu, of, first));
            const bool here = sg.tile0() >= c_lo && sg.end() <= c_hi;
            const int32_t g = sg.sub / row_groups, row0 = (sg.sub - g * row_groups) * R;
            Group x;
            x.first = __popc(valid & ((1u << first) - 1));
            x.n = __popc(set);
            x.rows = min(R, m.group - row0);
            x.out = here ? -1 : sg.tile0() >= c_lo;
            x.h = (int64_t)sg.b * m.hq + g * m.group + row0;
            if (lane == 0) group[k] = x;
            // Weights: a lane has one row of every (32 / R)-th part.
            constexpr int kSub = 32 / R, kEach = (2 * W + kSub - 1) / kSub;
            const int row = lane % R;
            float pm[kEach], pl[kEach], mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = i * kSub + lane / R;
                const bool in = at < 2 * W && (set >> at & 1);
                pm[i] = in ? part[at].m[row] : -INFINITY;
                pl[i] = in ? part[at].l[row] : 0.f;
                mm = fmaxf(mm, pm[i]);
            }
#pragma unroll
            for (int s = 16; s >= R; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = i * kSub + lane / R;
                const float w = pm[i] == -INFINITY ? 0.f : ex2_approx(pm[i] - mm);
                if (at < 2 * W && (set >> at & 1)) weight[__popc(valid & ((1u << at) - 1))][row] = w;
                ll += w * pl[i];
            }
#pragma unroll
            for (int s = 16; s >= R; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
            if (lane < x.rows) {
                if (here) {
                    lse[x.h + row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * (1.f / kLog2e);
                    scale_of[k][row] = ll == 0.f ? 0.f : 1.f / ll;
                } else {
                    mine[x.out].m[row] = mm, mine[x.out].l[row] = ll;
                }
            }
        }
    }
    __syncthreads();
    for (int x = tid; x < n_groups * R * kCols; x += kThreads) {
        const int k = x / (R * kCols), row = x / kCols % R, c = x % kCols * 4;
        const Group gr = group[k];
        if (row >= gr.rows) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = gr.first; i < gr.first + gr.n; ++i) {
            const float w = weight[i][row];
            const float4 z = *reinterpret_cast<const float4*>(&part[list[i]].o[row][c]);
            acc.x += w * z.x, acc.y += w * z.y, acc.z += w * z.z, acc.w += w * z.w;
        }
        if (gr.out >= 0) {
            *reinterpret_cast<float4*>(&mine[gr.out].o[row][c]) = acc;
        } else if (c < m.d) {
            const float inv = scale_of[k][row];
            store4(o + (gr.h + row) * m.d + c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
    }

    // ---- join the blocks' parts: the last block of a segment to arrive
    if (side[0].n + side[1].n == 0) return;
    __threadfence();
    __syncthreads();
    if (tid < 2 && side[tid].n) {
        // Counts up to the number of blocks and wraps to 0 by itself: ready for the next call. A block that skipped
        // its work for the status word's sake arrives all the same.
        const uint32_t n = side[tid].n;
        side[tid].last = atomicInc(counters + side[tid].first, n - 1) == n - 1 && !skip;
    }
    __syncthreads();
    for (int sd = 0; sd < 2; ++sd) {
        const Side S = side[sd];
        if (!S.last) continue;
        __threadfence();
        // Block k's part; only the first block leaves the segment, the others entered it.
        const P* all = reinterpret_cast<const P*>(slots) + 2 * S.first;
        float* wt = reinterpret_cast<float*>(smem);  // [n][R]: maxima, then weights
        float* ls = wt + kMaxParts * R;              // [n][R]: sums
        float* inv = ls + kMaxParts * R;             // [R]
        // The first parts' values are asked for before their weights are known.
        constexpr int kAhead = 16;
        float4 z[kAhead];
        auto load = [&](int x, int k0) {
            const float* p = &all[2 * k0].o[0][0] + x * 4;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                z[k] = x < S.rows * kCols && k0 + k < S.n
                           ? __ldcg(reinterpret_cast<const float4*>(p + (2 * k + (k0 + k == 0)) * (sizeof(P) / 4)))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        load(tid, 0);
        for (int x = tid; x < S.n * R; x += kThreads) {
            const int k = x / R, row = x % R;
            if (row >= S.rows) continue;
            wt[x] = __ldcg(&all[2 * k + (k == 0)].m[row]);
            ls[x] = __ldcg(&all[2 * k + (k == 0)].l[row]);
        }
        __syncthreads();
        for (int row = warp; row < S.rows; row += W) {
            float mm = -INFINITY, ll = 0.f;
            for (int k = lane; k < S.n; k += 32) mm = fmaxf(mm, wt[k * R + row]);
#pragma unroll
            for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
            for (int k = lane; k < S.n; k += 32) {
                const float pm = wt[k * R + row], w = pm == -INFINITY ? 0.f : ex2_approx(pm - mm);
                wt[k * R + row] = w;
                ll += w * ls[k * R + row];
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, x);
            if (lane == 0) {
                inv[row] = ll == 0.f ? 0.f : 1.f / ll;
                lse[S.h + row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * (1.f / kLog2e);
            }
        }
        __syncthreads();
        for (int x = tid; x < S.rows * kCols; x += kThreads) {
            const int row = x / kCols, c = x % kCols * 4;
            if (x != tid) load(x, 0);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < S.n; k0 += kAhead) {
                if (k0) load(x, k0);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float w = k0 + k < S.n ? wt[(k0 + k) * R + row] : 0.f;
                    acc.x += w * z[k].x, acc.y += w * z[k].y, acc.z += w * z[k].z, acc.w += w * z[k].w;
                }
            }
            const float i = inv[row];
            if (c < m.d) store4(o + (S.h + row) * m.d + c, make_float4(acc.x * i, acc.y * i, acc.z * i, acc.w * i));
        }
        __syncthreads();  // the weights have been read
    }
}

// One compiled kernel: type, channels (rounded up), tiles of 8 query rows and warps of a block.
template <typename T_, int DP_, int NT_, int W_>
struct Variant {
    using T = T_;
    static constexpr int DP = DP_, NT = NT_, W = W_;
    using P = Partial<DP, 8 * NT>;
    static constexpr size_t kWorkspace = kCounterBytes + sizeof(P) * kMaxParts * 2;
    static constexpr size_t kShared = sizeof(P) * W * 2 + Frag<T, DP, NT>::kShared * 512 * W;
};

// fn(variant) with the variant for a cache: the scratch's size and the launch come from the same choice. `units`: the most
// units an SM may get, by the shapes; `listed`: of pages in a list. Variants that these choose between differ in warps
// only, which the scratch does not see.
//   More than 8 query heads a kv head: 16 rows a warp read K and V once (4 x 60000 keys, 32/2 heads, d 128: 58 us; 8 rows
//   a warp, the second half from L2: 66 us). float32 has no registers for 16 rows; at 8 rows and d 128 it spills 60 bytes.
//   Warps: as many as leave the registers for a tile of K and of V in flight (d 64, 8 rows: 12 warps 51 us, 16 warps
//   of fewer registers 57 us; 16 rows: 12 warps 36 us, 8 warps 40 us. d 128, 16 rows: 8 warps, which spill
//   24 bytes, 58 us, 10 spill more, 96 us).
//   Where there is little to read, 8, if there is a choice (up to 8 rows, bf16 d 128 and float32 d 64): fewer parts to join,
//   no spills (d 128, 4 kv heads: 1000 keys 13.1 us with 12
//   warps, 11.7 with 8; 32768 keys, 55 units an SM, 23.9 and 22.5; 2 x 60000 keys, 203, 50.0 and 49.8; 8 x 131071, 1771,
//   322 and 330. float32, d 64, 4 kv heads: 27 units 17.6 and 16.7; 55, 27.4 and 27.9; 101, 38.5 and 41.6). A list of pages
//   is one more load to wait for, which more warps hide (select and decode of 200 pages of 16 positions, 4 kv heads: 43
//   units 43.6 us with 12 warps, 42.4 with 8; 86, 60.1 and 59.8; 173, 84 and 89).
// "Little to read" goes by the table's width, as lengths are device data: a table that is far wider than its sequences are
// long gets 12 warps for them (1000 keys, 4 kv heads: 11.3 us with a table of 63 or 4096 pages, 12.8 with 65536; 333 keys
// 9.9 and 10.9; 8 x 1000 keys, 8 kv heads, 18.4 and 20.0 from 4096 pages on).
constexpr int64_t kFewBf16 = 400, kFewBf16Listed = 80, kFewF32 = 40;

template <typename F>
auto with_variant(const PagedMeta& m, int64_t units, bool listed, F&& fn) {
    using B = __nv_bfloat16;
    if (m.dtype == SPLITKV_F32) {
        if (m.d > 64) return fn(Variant<float, 128, 1, 8>{});
        return units <= kFewF32 ? fn(Variant<float, 64, 1, 8>{}) : fn(Variant<float, 64, 1, 12>{});
    }
    if (m.group > 8) return m.d <= 64 ? fn(Variant<B, 64, 2, 12>{}) : fn(Variant<B, 128, 2, 8>{});
    if (m.d <= 64) return fn(Variant<B, 64, 1, 12>{});
    return units <= (listed ? kFewBf16Listed : kFewBf16) ? fn(Variant<B, 128, 1, 8>{}) : fn(Variant<B, 128, 1, 12>{});
}

}  // namespace

size_t paged_decode_workspace(const PagedMeta& m) {
    return with_variant(m, 0, false, [](auto v) { return decltype(v)::kWorkspace; });
}

int64_t paged_decode_units(const PagedMeta& m) {
    const int64_t tiles = ((int64_t)m.max_pages * m.page + kTile - 1) / kTile;
    return (tiles + kSegmentCost) * m.hkv * ((m.group + 7) / 8);
}

namespace {

cudaError_t launch_some(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                        const int32_t* table, const int32_t* seq_len, const int32_t* pages, int32_t n_select, void* o,
                        float* lse, int32_t* status, void* ws, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t positions = (int64_t)(pages ? std::min(n_select, m.max_pages) : m.max_pages) * m.page;
    const int64_t rows = (int64_t)m.n_seqs * m.hkv * ((m.group + 7) / 8);
    return with_variant(m, rows * ((positions + kTile - 1) / kTile) / sms, pages != nullptr, [&](auto v) {
        using V = decltype(v);
        using T = typename V::T;
        auto kern = decode_kernel<T, V::DP, V::NT, V::W>;
        static SmemGrants granted;
        const cudaError_t e =
            allow_smem((const void*)kern, V::kShared + sizeof(int32_t) * (SPLITKV_PAGED_MAX_SEQS + 1), granted);
        if (e != cudaSuccess) return e;
        const size_t smem = V::kShared + sizeof(int32_t) * std::max(m.n_seqs + 1, V::W * 36);
        return note_error(launch_overlapped(kern, std::min(sms, kMaxParts), V::W * 32, smem, st, m, (const T*)q, q_stride,
                                            (const T*)k_cache, (const T*)v_cache, table, seq_len, pages, n_select, (T*)o,
                                            lse, status, (uint32_t*)ws, (char*)ws + kCounterBytes),
                          "paged decode");
    });
}

}  // namespace

cudaError_t launch_paged_decode(const PagedMeta& m, const void* q, int64_t q_stride, const void* k_cache,
                                const void* v_cache, const int32_t* table, const int32_t* seq_len,
                                const int32_t* pages, int32_t n_select, void* o, float* lse, int32_t* status, void* ws,
                                cudaStream_t st) {
    const int32_t most = (int32_t)(INT32_MAX / paged_decode_units(m));
    const int64_t size = m.dtype == SPLITKV_BF16 ? 2 : 4;
    for (int32_t b = 0; b < m.n_seqs; b += most) {
        PagedMeta some = m;
        some.n_seqs = std::min(most, m.n_seqs - b);
        const cudaError_t e =
            launch_some(some, (const char*)q + b * q_stride * size, q_stride, k_cache, v_cache, table + b * m.table_stride,
                        seq_len + b, pages ? pages + (int64_t)b * m.hkv * n_select : nullptr, n_select,
                        (char*)o + (int64_t)b * m.hq * m.d * size, lse + (int64_t)b * m.hq, status, ws, st);
        if (e != cudaSuccess || most >= m.n_seqs - b) return e;
    }
    return cudaSuccess;
}

}  // namespace splitkv
