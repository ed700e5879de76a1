// Matrix products of the dense layers (gnn_linear, gnn_gated_linear and their backward passes): the
// tiled kernel, its operand orders and its epilogue.  Internal; instantiated by dense_bf16.hip and
// dense_f32.hip, planned by dense.hip.
//
// One kernel serves the three products of a layer y = x W, x [n, d_in], W [d_in, d_out]:
//   forward   y  = x W        rows of x, summed index contiguous;  W, summed index strided
//   gradient  dx = dz W^T     rows of dz, contiguous;              W, contiguous
//   gradient  dW = x^T dz     x, strided;                          dz, strided
// The left operand gives the rows of the product ("A"), the right one its columns ("B").  A product may
// be a sum over segments, each with operands of its own (the two projections of a gated layer, the two
// planes of a rounded gradient).
//
// Matrix instructions are 32 x 32 (16 summed for bf16, 2 for fp32).  B is their first operand, so that a
// lane holds one row of the product, and the columns of B are dealt to the instruction's rows so that the
// 16 values a lane holds lie next to each other: the epilogue loads and stores 32 or 64 bytes a lane.
//
// LDS holds a tile of 128 bytes of the summed index (64 bf16, 32 fp32) a row or column, in NB buffers.
// Contiguous operands lie in rows of eight 16-byte pieces; strided ones as in memory, one line of the
// tile's width per summed index, and the matrix instruction's operand is turned on the way out of LDS
// (ds_read_b64_tr_b16; fp32 takes single words).  Pieces are permuted within their line so that what one
// LDS read touches spreads over the banks: lds_piece below.  Where both operands start at multiples of 16
// bytes and their lines are whole pieces, tiles go from memory into LDS directly (kDirect); otherwise
// through registers.  A tile that the summed length cuts is filled with zeros, element by element where
// it must be.
#pragma once

#include "learn.hpp"

namespace gnnmb {

// Order of the operands' elements, see above.
enum : int32_t { kForward, kGradX, kGradW };

// What becomes of a sum z = A B (of both sums g, u of a gated layer).
struct Epilogue {
    int32_t act;
    const void *bias[2];                // [cols], may be NULL
    const void *res;                    // [rows, ld_res], may be NULL: added last
    int64_t ld_res;
    void *pre[2];                       // [rows, ld_pre]: z (g and u) as they are, may be NULL
    int64_t ld_pre;
    void *out[2];                       // [rows, ld_out]: act(z) + res, or act(g) u in out[0]
    int64_t ld_out;
};

struct ProductArgs {
    const void *a[4];                   // of each segment
    const void *b[2][4];                // of each product of the launch (or each of a pair) and segment
    int64_t ld_a, ld_b;
    int64_t rows, cols, k;              // k: of one segment
    const int64_t *d_n;                 // NULL, or how many of the rows (kGradW: of k) count
    int32_t segs;
    int32_t short_segs;                 // segments where fewer than kShortSum of k count
    int32_t products;                   // products of the launch (one where it is a gated pair)
    int32_t splits;                     // parts of the summed length, whose sums go to part
    int64_t r_tiles, c_tiles, first_tile;     // set by the launcher
    float *part;                        // [splits][products or pair][rows][ld_part], or NULL: the epilogue follows
    int64_t ld_part;
    Epilogue e;
};

// A rounding of a summed operand to bf16 is as large as the result's own rounding where few terms are
// summed: below this many, the gradients dz are taken in two planes (see dense.hip).
constexpr int64_t kShortSum = 512;

// ---- activations ----------------------------------------------------------------------------------

// exp and reciprocal of the bf16 kernels: a few 2^-23 off, against the 2^-9 of the result's rounding.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
    if (FAST) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.442695041f * z));
    return 1.f / (1.f + expf(-z));
}

// Lower tail of the normal distribution, Phi(z) = erfc(-z / sqrt 2) / 2, and e^(-z^2 / 2).  The fast form
// is exp(-a^2) times a polynomial in t = 1 / (1 + a / 2) for a = |z| / sqrt 2, fitted to
// erfc(a) exp(a^2) at Chebyshev points with weights 1 / value: relative error 1.3e-5 over all a.
template <bool FAST>
__device__ __forceinline__ float normal_tail(float z, float *bell) {
    if (!FAST) {
        *bell = expf(-0.5f * z * z);
        return 0.5f * erfcf(-0.70710678f * z);
    }
    const float e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
    *bell = e;
    const float t = __builtin_amdgcn_rcpf(1.f + 0.35355339f * __builtin_fabsf(z));
    const float q = e * t * ((((((0.0285215937f * t + -0.127408415f) * t + 0.129590943f) * t + 0.0598448329f) *
                        t + 0.127570897f) * t + 0.140824407f) * t + 0.1410494f);
    return z < 0.f ? q : 1.f - q;
}

template <bool FAST, int V>
__device__ __forceinline__ vec<float, V> activate(int32_t act, vec<float, V> z) {
    float bell;
    switch (act) {
    case GNN_ACT_RELU:
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] > 0.f || z[i] != z[i] ? z[i] : 0.f;
        break;
    case GNN_ACT_GELU:
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= normal_tail<FAST>(z[i], &bell);
        break;
    case GNN_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= sigmoid<FAST>(1.595769122f * (z[i] + 0.044715f * z[i] * z[i] * z[i]));
        break;
    case GNN_ACT_SILU:
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= sigmoid<FAST>(z[i]);
        break;
    case GNN_ACT_SIGMOID:
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = sigmoid<FAST>(z[i]);
        break;
    default:
        break;
    }
    return z;
}

// act(z) (in z) and act'(z).
template <bool FAST, int V>
__device__ __forceinline__ vec<float, V> activate_slope(int32_t act, vec<float, V> &z) {
    vec<float, V> s(1.f);
    switch (act) {
    case GNN_ACT_RELU:
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = z[i] > 0.f ? 1.f : 0.f;
            z[i] = z[i] > 0.f || z[i] != z[i] ? z[i] : 0.f;
        }
        break;
    case GNN_ACT_GELU:
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float bell;
            const float y = normal_tail<FAST>(z[i], &bell);
            s[i] = y + 0.39894228f * z[i] * bell;
            z[i] *= y;
        }
        break;
    case GNN_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float zz = z[i] * z[i];
            const float y = sigmoid<FAST>(1.595769122f * z[i] * (1.f + 0.044715f * zz));
            s[i] = y + z[i] * y * (1.f - y) * (1.595769122f + 0.2140644488f * zz);
            z[i] *= y;
        }
        break;
    case GNN_ACT_SILU:
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float y = sigmoid<FAST>(z[i]);
            s[i] = y * (1.f + z[i] * (1.f - y));
            z[i] *= y;
        }
        break;
    case GNN_ACT_SIGMOID:
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = sigmoid<FAST>(z[i]);
            s[i] = z[i] * (1.f - z[i]);
        }
        break;
    default:
        break;
    }
    return s;
}

// ---- epilogue ---------------------------------------------------------------------------------------

// The first `count` of V elements (all of them in one piece where that many exist).
template <typename T, int V>
__device__ __forceinline__ vec<float, V> load_some(const T *p, int64_t count) {
    if (count >= V) return load_f32<T, V>(p);
    vec<float, V> v(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < count) v[i] = static_cast<float>(p[i]);
    return v;
}

template <typename T, int V>
__device__ __forceinline__ void store_some(T *p, int64_t count, vec<float, V> v) {
    if (count >= V) {
        store_f32<T, V>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < count) p[i] = static_cast<T>(v[i]);
}

// V values of row m from column n on, `count` of which exist; PAIR: v and u are a gated layer's sums.
template <typename T, int V, bool PAIR>
__device__ __forceinline__ void finish(const Epilogue &e, int z, int64_t m, int64_t n, int64_t count,
                                       vec<float, V> v, vec<float, V> u) {
    constexpr bool kFast = sizeof(T) == 2;
    if (e.bias[z]) v += load_some<T, V>(static_cast<const T *>(e.bias[z]) + n, count);
    if (e.pre[z]) store_some<T, V>(static_cast<T *>(e.pre[z]) + m * e.ld_pre + n, count, v);
    v = activate<kFast, V>(e.act, v);
    if (PAIR) {
        if (e.bias[1]) u += load_some<T, V>(static_cast<const T *>(e.bias[1]) + n, count);
        if (e.pre[1]) store_some<T, V>(static_cast<T *>(e.pre[1]) + m * e.ld_pre + n, count, u);
        v *= u;
    }
    if (e.res) v += load_some<T, V>(static_cast<const T *>(e.res) + m * e.ld_res + n, count);
    store_some<T, V>(static_cast<T *>(e.out[z]) + m * e.ld_out + n, count, v);
}

// ---- tiles ------------------------------------------------------------------------------------------

typedef vec<uint32_t, 4> u4;
typedef vec<uint32_t, 2> u2;
typedef vec<float, 16> f16x;

// Row or column of an operand's 32 that the matrix instruction's index r stands for.  For B it deals
// r = 8 g + 4 h + e to 16 h + 4 g + e: a lane of half h holds r = 8 g + 4 h + 0..3 for g = 0..3.
template <bool B>
__device__ __forceinline__ int dealt(int r) {
    return B ? ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3) : r;
}

// Which piece of memory line r (contiguous operands: the row or column, eight pieces; strided ones: the
// summed index, CPR pieces) lies at place c of LDS line r; an involution in c.
//  - Contiguous: one read takes the same piece of 32 lines, in the order of dealt; eight lanes of it cover
//    128 bytes, sixteen 256 (the parity of the line gives the half).
//  - Strided bf16: sixteen lanes read 4 lines of the summed index and, of each, two pieces: next to each
//    other for A, one apart for B; 32 lanes four pieces in a row.
//  - Strided fp32: 32 lanes read 128 bytes of one line, the others of the line four below.
template <typename T, bool CONTIGUOUS, bool B, int CPR>
__device__ __forceinline__ int lds_piece(int r, int c) {
    if (CONTIGUOUS) {
        const int low = B ? ((r >> 4) & 1) * 4 + (r & 3) : r & 7;
        return c ^ low ^ ((B ? r >> 2 : r >> 3) & 1);
    }
    if (sizeof(T) == 4) return c ^ ((r >> 2) & 1) * 8;
    if (CPR == 8) return c ^ ((r & 1) | (r & 2) << 1);
    return c ^ ((r & 1) * 4 | ((r >> 1) & 1) * 11);
}

// A load from memory into LDS: 16 bytes of each lane, from base + offset, to 16 bytes times the lane
// from `lds` on (both uniform).  It writes no register; vmcnt counts it, but the compiler does not (of the
// builtin it knows, and waits for all of them before every read of LDS that it cannot tell apart).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"      // that m0 is reserved
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const void *base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

template <int PENDING>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(PENDING) : "memory");
}

typedef __attribute__((address_space(3))) char lds_char;

template <typename T>
struct Step;     // one step of the tile's four: 16 bytes of the summed index per lane and operand

template <>
struct Step<bf16> {
    static constexpr int kElems = 8;
    static __device__ __forceinline__ f16x mul(u4 b, u4 a, f16x c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(vec<bf16, 8>, b),
                                                       __builtin_bit_cast(vec<bf16, 8>, a), c, 0, 0, 0);
    }
};

template <>
struct Step<float> {
    static constexpr int kElems = 4;
    static __device__ __forceinline__ f16x mul(u4 b, u4 a, f16x c) {
        const vec<float, 4> x = __builtin_bit_cast(vec<float, 4>, b), y = __builtin_bit_cast(vec<float, 4>, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
        return c;
    }
};

// TILE lines of one operand for a product tile: what the threads load of it and where a wavefront reads.
// SUB: column stretches of their own (two for the pair of a gated layer), TILE / SUB wide each.
template <typename T, bool CONTIGUOUS, bool B, int TILE, int SUB, int THREADS>
struct TileOf {
    static constexpr int kElems = Step<T>::kElems;
    static constexpr int kWide = TILE / SUB;
    static constexpr int kCpr = CONTIGUOUS ? 8 : kWide / kElems;      // pieces per LDS line
    static constexpr int kPieces = TILE * 8 / THREADS;                // pieces per thread
    static constexpr int kBytes = TILE * 128;
    static constexpr int kLinesPerPass = THREADS / kCpr;
    static_assert(kPieces % SUB == 0 && kPieces > 0, "a pass of the threads lies in one stretch");
    static_assert(CONTIGUOUS ? kLinesPerPass % 32 == 0 : kLinesPerPass % 8 == 0, "lds_piece repeats from pass to pass");

    // Line and memory piece of this thread's piece i (within its stretch).
    static __device__ __forceinline__ int line(int i, int t) { return (i % (kPieces / SUB)) * kLinesPerPass + t / kCpr; }
    static __device__ __forceinline__ int piece(int t) {
        return lds_piece<T, CONTIGUOUS, B, kCpr>(t / kCpr, t % kCpr);
    }

    // Byte offsets of the thread's loads from the operand's start (strided: from the summed index's line).
    // Lines or columns beyond `limit` repeat the last ones; what they give is not stored.
    static constexpr int kOffsets = CONTIGUOUS ? kPieces : 1;
    uint32_t offset[kOffsets];
    int64_t first;          // contiguous: first line of the tile
    int64_t limit;
    int shift;              // strided: elements by which a piece at the lines' end is moved

    __device__ __forceinline__ void init(int64_t first_, int64_t limit_, int64_t ld, int t) {
        first = first_;
        limit = limit_;
        shift = 0;
        if (CONTIGUOUS) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                int64_t r = line(i, t);
                if (first + r >= limit) r = limit - 1 - first;
                offset[i] = static_cast<uint32_t>(r * ld + piece(t) * kElems) * static_cast<uint32_t>(sizeof(T));
            }
        } else {
            int64_t c = first + piece(t) * kElems;
            const int64_t last = limit < kElems ? 0 : limit - kElems;
            if (c > last) {
                if (c < limit) shift = static_cast<int>(c - last);
                c = last;
            }
            offset[0] = static_cast<uint32_t>(c + t / kCpr * ld) * static_cast<uint32_t>(sizeof(T));
        }
    }
    // Start of the loads of piece i for summed index k0.
    __device__ __forceinline__ const char *base(const void *p, int64_t ld, int i, int64_t k0) const {
        const int64_t e = CONTIGUOUS ? first * ld + k0 : (k0 + (i % (kPieces / SUB)) * kLinesPerPass) * ld;
        return static_cast<const char *>(p) + e * static_cast<int64_t>(sizeof(T));
    }
    __device__ __forceinline__ uint32_t at(int i) const { return offset[CONTIGUOUS ? i : 0]; }

    // One piece, with zeros where the summed length k or the limit ends.
    __device__ __forceinline__ u4 cut(const void *from, int64_t ld, int i, int64_t k0, int64_t k, int t) const {
        const T *p = static_cast<const T *>(from);
        int64_t there;
        if (CONTIGUOUS) {
            int64_t r = first + line(i, t);
            if (r >= limit) r = limit - 1;
            const int64_t c = k0 + piece(t) * kElems;
            p += r * ld + c;
            there = k - c;
        } else {
            const int64_t r = k0 + line(i, t), c = first + piece(t) * kElems;
            p += r * ld + c;
            there = r < k ? limit - c : 0;
        }
        vec<T, kElems> v(static_cast<T>(0.f));
        if (there >= kElems) {
            v = *reinterpret_cast<const typename loose<T, kElems>::type *>(p);
        } else {
#pragma unroll
            for (int e = 0; e < kElems; ++e)
                if (e < there) v[e] = p[e];
        }
        return __builtin_bit_cast(u4, v);
    }
    // A piece that was loaded `shift` elements too early, put right.
    __device__ __forceinline__ u4 shifted(u4 v) const {
        if (shift == 0) return v;
        unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
        return __builtin_bit_cast(u4, x >> (shift * 8 * static_cast<int>(sizeof(T))));
    }

    // Where in LDS a lane's 16 bytes of 32 lines `frag` lie for step 0 of a tile, in bytes.
    static __device__ __forceinline__ uint32_t read_base(int frag, int lane) {
        const int half = lane >> 5;
        if (CONTIGUOUS) {
            const int r = dealt<B>(lane & 31);
            return (frag * 32 + r) * 128 + lds_piece<T, true, B, 8>(r, half) * 16;
        }
        if (sizeof(T) == 4) {
            const int c = frag * 32 + dealt<B>(lane & 31), r = half * 4;
            return r * kWide * 4 + lds_piece<T, false, B, kCpr>(r, c >> 2) * 16 + (c & 3) * 4;
        }
        // sixteen lanes give the four columns' lines of four summed indices each
        const int r = half * 8 + ((lane & 15) >> 2);
        const int c = frag * 32 + dealt<B>(((lane >> 4) & 1) * 16 + (lane & 3) * 4);
        return r * kWide * 2 + lds_piece<T, false, B, kCpr>(r, c >> 3) * 16 + (c & 4) * 2;
    }
    static __device__ __forceinline__ u4 read(const lds_char *lds, uint32_t base, int step) {
        if (CONTIGUOUS)       // the step's two pieces: bits 5 and 6 of a place's address
            return *reinterpret_cast<const __attribute__((address_space(3))) u4 *>(lds + (base ^ (step * 32)));
        if constexpr (sizeof(T) == 4) {
            u4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t *>(
                    lds + base + (step * 8 + i) * kWide * 4);
            return v;
        } else {
            typedef vec<short, 4> s4;
            typedef __attribute__((address_space(3))) s4 lds_s4;
            lds_char *p = const_cast<lds_char *>(lds) + base + step * 16 * kWide * 2;
            const u2 lo = __builtin_bit_cast(
                u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4 *>(p)));
            const u2 hi = __builtin_bit_cast(
                u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4 *>(p + 4 * kWide * 2)));
            return u4{lo[0], lo[1], hi[0], hi[1]};
        }
    }
};

// ---- the product ------------------------------------------------------------------------------------

template <typename T, int FORM, int TR, int TC, int WR, int WC, int NB, int WAVES, bool PAIR, bool DIRECT>
__global__ __launch_bounds__(WR * WC * 64, WAVES) void k_product(ProductArgs p) {
    constexpr int kThreads = WR * WC * 64;
    constexpr int kBk = 128 / static_cast<int>(sizeof(T));
    constexpr int FR = TR / WR / 32, FC = TC / WC / 32;       // 32 x 32 sums of a wavefront
    static_assert(FR > 0 && FC > 0 && (!PAIR || FC % 2 == 0), "a wavefront holds both sums of a pair");
    static_assert(DIRECT || NB == 2, "through registers: one tile under way");
    typedef TileOf<T, FORM != kGradW, false, TR, 1, kThreads> A;
    typedef TileOf<T, FORM == kGradX, true, TC, PAIR ? 2 : 1, kThreads> B;
    constexpr int kPieces = A::kPieces + B::kPieces;
    constexpr int kBuffer = A::kBytes + B::kBytes;
    __shared__ __align__(1024) char lds[NB * kBuffer];
    lds_char *const shared = (lds_char *)lds;

    // The tile, and the part of the summed length, of this workgroup.  Workgroups b, b + 8, ... run on one
    // XCD: each XCD takes a stretch of tiles next to each other, whose lines its L2 then holds; the tiles go
    // in columns of eight, so that a stretch is about as high as wide.
    constexpr int64_t kXcds = 8, kHigh = 8;
    const int64_t tiles = p.r_tiles * p.c_tiles;
    int64_t q = p.first_tile + blockIdx.x;
    const int64_t outer = q / tiles;                        // split, product
    q -= outer * tiles;
    const int64_t whole = tiles / kXcds * kXcds;
    if (q < whole) q = q % kXcds * (whole / kXcds) + q / kXcds;
    const int64_t per = kHigh * p.c_tiles, g = q / per, in = q - g * per;
    const int64_t high = p.r_tiles - kHigh * g < kHigh ? p.r_tiles - kHigh * g : kHigh;
    const int64_t tc = in / high, tr = kHigh * g + in - tc * high;
    const int z = static_cast<int>(outer % p.products);
    const int64_t split = outer / p.products;

    const int64_t rows = FORM == kGradW ? p.rows : load_count(p.d_n, p.rows);
    const int64_t k = FORM == kGradW ? load_count(p.d_n, p.k) : p.k;
    const int64_t r0 = tr * TR, c0 = tc * (PAIR ? TC / 2 : TC);
    if (r0 >= rows) return;      // whole workgroup

    const int t = threadIdx.x, lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wr = w / WC, wc = w % WC;
    A ta;
    B tb;
    ta.init(r0, rows, p.ld_a, t);
    tb.init(c0, p.cols, p.ld_b, t);

    const int64_t seg_tiles = (k + kBk - 1) / kBk;
    const int segs = k < kShortSum ? p.short_segs : p.segs;
    int64_t lo = 0, steps64 = seg_tiles * segs;
    if (p.splits > 1) {
        const int64_t share = (steps64 + p.splits - 1) / p.splits;
        lo = split * share < steps64 ? split * share : steps64;
        steps64 = steps64 - lo < share ? steps64 - lo : share;
    }
    const int steps = static_cast<int>(steps64);
    // segment and summed index of the next tile to load
    int seg = seg_tiles > 0 ? static_cast<int>(lo / seg_tiles) : 0;
    int64_t k0 = (lo - seg * seg_tiles) * kBk;

    // A tile narrower than a piece is always taken element by element.
    const bool narrow = !DIRECT && ((FORM == kGradW && p.rows < A::kElems) || (FORM != kGradX && p.cols < B::kElems));
    u4 ra[DIRECT ? 1 : A::kPieces], rb[DIRECT ? 1 : B::kPieces];
    bool staged = false;       // the tile that was last issued waits in ra and rb
    const uint32_t lds0 = static_cast<uint32_t>((uintptr_t)shared);
    auto issue = [&](int buf) {
        const void *pa = p.a[seg];
        const void *pb0 = p.b[z][seg], *pb1 = PAIR ? p.b[1][seg] : nullptr;
        if (k0 + kBk <= k && !narrow) {
            if (DIRECT) {
                const uint32_t to = lds0 + buf * kBuffer + w * 1024;
#pragma unroll
                for (int i = 0; i < A::kPieces; ++i)
                    load_to_lds(to + i * kThreads * 16, ta.at(i), ta.base(pa, p.ld_a, i, k0));
#pragma unroll
                for (int i = 0; i < B::kPieces; ++i)
                    load_to_lds(to + A::kBytes + i * kThreads * 16, tb.at(i),
                                tb.base(PAIR && i >= B::kPieces / 2 ? pb1 : pb0, p.ld_b, i, k0));
            } else {
                staged = true;
#pragma unroll
                for (int i = 0; i < A::kPieces; ++i)
                    ra[i] = __builtin_bit_cast(u4, *reinterpret_cast<const typename loose<T, A::kElems>::type *>(
                                                       ta.base(pa, p.ld_a, i, k0) + ta.at(i)));
#pragma unroll
                for (int i = 0; i < B::kPieces; ++i)
                    rb[i] = __builtin_bit_cast(u4, *reinterpret_cast<const typename loose<T, B::kElems>::type *>(
                                                       tb.base(PAIR && i >= B::kPieces / 2 ? pb1 : pb0, p.ld_b, i, k0) + tb.at(i)));
            }
        } else {
            staged = false;
            u4 *to = reinterpret_cast<u4 *>(lds + buf * kBuffer) + t;
            for (int i = 0; i < A::kPieces; ++i) to[i * kThreads] = ta.cut(pa, p.ld_a, i, k0, k, t);
            to += A::kBytes / 16;
            for (int i = 0; i < B::kPieces; ++i)
                to[i * kThreads] = tb.cut(PAIR && i >= B::kPieces / 2 ? pb1 : pb0, p.ld_b, i, k0, k, t);
        }
        k0 += kBk;
        if (k0 >= k) {
            k0 = 0;
            ++seg;
        }
    };
    // Through registers: the tile that was last issued goes into LDS.
    const bool turned = !DIRECT && (p.rows % A::kElems != 0 || p.cols % B::kElems != 0);
    auto commit = [&](int buf) {
        if (DIRECT || !staged) return;
        u4 *to = reinterpret_cast<u4 *>(lds + buf * kBuffer) + t;
        if (turned) {
#pragma unroll
            for (int i = 0; i < A::kPieces; ++i) ra[i] = ta.shifted(ra[i]);
#pragma unroll
            for (int i = 0; i < B::kPieces; ++i) rb[i] = tb.shifted(rb[i]);
        }
#pragma unroll
        for (int i = 0; i < A::kPieces; ++i) to[i * kThreads] = ra[i];
#pragma unroll
        for (int i = 0; i < B::kPieces; ++i) to[A::kBytes / 16 + i * kThreads] = rb[i];
    };

    f16x acc[FR][FC];
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int j = 0; j < FC; ++j) acc[i][j] = f16x(0.f);
    uint32_t at_a[FR], at_b[FC];
#pragma unroll
    for (int i = 0; i < FR; ++i) at_a[i] = A::read_base(wr * FR + i, lane);
#pragma unroll
    for (int j = 0; j < FC; ++j)
        at_b[j] = A::kBytes + (PAIR ? (j & 1) * (B::kBytes / 2) + B::read_base(wc * (FC / 2) + j / 2, lane)
                                    : B::read_base(wc * FC + j, lane));
    u4 fa[2][FR], fb[2][FC];
    auto read = [&](int buf, int step, int at) {
        const lds_char *from = shared + buf * kBuffer;
        if (at < FR)
            fa[step & 1][at] = A::read(from, at_a[at], step);
        else
            fb[step & 1][at - FR] = B::read(from, at_b[at - FR], step);
    };
    constexpr int kReads = FR + FC, kProducts = FR * FC;
    // The products of a step, and between them the reads of the next.
    auto multiply = [&](int step, bool next, int buf, int next_step) {
#pragma unroll
        for (int ij = 0; ij < kProducts; ++ij) {
            const int i = ij / FC, j = ij % FC;
            acc[i][j] = Step<T>::mul(fb[step & 1][j], fa[step & 1][i], acc[i][j]);
            if (next) {
#pragma unroll
                for (int r = ij * kReads / kProducts; r < (ij + 1) * kReads / kProducts; ++r) read(buf, next_step, r);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    if (steps > 0) {
        if (DIRECT) {
#pragma unroll
            for (int j = 0; j < NB - 1; ++j)
                if (j < steps) issue(j);
            if (steps >= NB - 1)
                wait_and_meet<(NB - 2) * kPieces>();
            else
                wait_and_meet<0>();
            if (NB - 1 < steps) issue(NB - 1);
        } else {
            issue(0);
            commit(0);
            wait_and_meet<0>();
            if (steps > 1) issue(1);
        }
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(0, 0, r);
        int buf = 0;
        for (int s = 0; s + 1 < steps; ++s) {
            const int next = buf + 1 == NB ? 0 : buf + 1;
#pragma unroll
            for (int step = 0; step < 3; ++step) multiply(step, true, buf, step + 1);
            // Tile s is read; the next one has to be there.
            commit(next);
            if (NB > 2 && s + NB <= steps)
                wait_and_meet<(NB - 2) * kPieces>();
            else
                wait_and_meet<0>();
            if (DIRECT) {
                if (s + NB < steps) issue(buf);
            } else {
                if (s + 2 < steps) issue(buf);
            }
            multiply(3, true, next, 0);
            buf = next;
        }
#pragma unroll
        for (int step = 0; step < 3; ++step) multiply(step, true, buf, step + 1);
        multiply(3, false, 0, 0);
    }

    // A lane holds row lane % 32 of each 32 x 32 sum, and its columns 16 (lane / 32) + 0..15.
#pragma unroll
    for (int i = 0; i < FR; ++i) {
        const int64_t m = r0 + (wr * FR + i) * 32 + (lane & 31);
        if (m >= rows) continue;
        const int left = lane >> 5 << 4;
#pragma unroll
        for (int j = 0; j < FC; j += PAIR ? 2 : 1) {
            const int64_t n = c0 + (PAIR ? wc * (FC / 2) + j / 2 : wc * FC + j) * 32 + left;
            if (n >= p.cols) continue;
            if (p.part) {
                const int64_t at = (split * (PAIR ? 2 : p.products) + z) * p.rows + m;
                store_some<float, 16>(p.part + at * p.ld_part + n, p.cols - n, acc[i][j]);
                if (PAIR) store_some<float, 16>(p.part + (at + p.rows) * p.ld_part + n, p.cols - n, acc[i][PAIR ? j + 1 : j]);
                continue;
            }
            finish<T, 16, PAIR>(p.e, z, m, n, p.cols - n, acc[i][j], acc[i][PAIR ? j + 1 : j]);
        }
    }
}

// ---- launching --------------------------------------------------------------------------------------

// Tile shapes of the kernel: 256 x 256 by eight wavefronts (bf16 only), 128 x 128 by four, 32 x 128 for
// few rows.
enum : int32_t { kTile256, kTile128, kTile32 };

struct ProductPlan {
    int32_t form, tile, pair, direct;
};

inline int tile_rows(int tile) { return tile == kTile256 ? 256 : tile == kTile128 ? 128 : 32; }
inline int tile_cols(int tile, bool pair) { return (tile == kTile256 ? 256 : 128) / (pair ? 2 : 1); }

hipError_t launch_product_bf16(ProductArgs a, const ProductPlan &p, hipStream_t s);
hipError_t launch_product_f32(ProductArgs a, const ProductPlan &p, hipStream_t s);

template <typename T, int FORM, int TR, int TC, int WR, int WC, int NB, int WAVES, bool PAIR, bool DIRECT>
hipError_t launch_tile(ProductArgs &a, hipStream_t s) {
    a.r_tiles = (a.rows + TR - 1) / TR;
    const int64_t wide = PAIR ? TC / 2 : TC;
    a.c_tiles = (a.cols + wide - 1) / wide;
    return launch_pieces(a.r_tiles * a.c_tiles * a.products * a.splits, WR * WC * 64, [&](int64_t first, unsigned blocks) {
        a.first_tile = first;
        k_product<T, FORM, TR, TC, WR, WC, NB, WAVES, PAIR, DIRECT><<<blocks, WR * WC * 64, 0, s>>>(a);
    });
}

template <typename T, int FORM, bool PAIR>
hipError_t launch_form(ProductArgs &a, const ProductPlan &p, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (p.tile == kTile256 && p.direct) return launch_tile<T, FORM, 256, 256, 2, 4, 2, 2, PAIR, true>(a, s);
    }
    if constexpr (FORM != kGradW && !PAIR) {
        if (p.tile == kTile32)
            return p.direct ? launch_tile<T, FORM, 32, 128, 1, 4, 4, 2, false, true>(a, s)
                            : launch_tile<T, FORM, 32, 128, 1, 4, 2, 2, false, false>(a, s);
    }
    return p.direct ? launch_tile<T, FORM, 128, 128, 2, 2, 2, 2, PAIR, true>(a, s)
                    : launch_tile<T, FORM, 128, 128, 2, 2, 2, 2, PAIR, false>(a, s);
}

}  // namespace gnnmb
