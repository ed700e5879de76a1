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
// LDS read touches spreads over the banks: lds_piece below.  Tiles go from memory into LDS directly, by
// pieces where both operands' lines start at multiples of 16 bytes and are whole pieces (kByPiece), by words
// where they are multiples of 4 bytes, fp32 always (kByWord); other bf16 operands go through registers
// (kThrough).  A tile that the summed length cuts is loaded through registers, shifted to its place and
// filled up with zeros.
//
// While the products of one tile run, those of the next NB - 1 are under way.  A barrier comes before the last of a
// tile's four steps, whose operands are in registers by then: the first reads of the next tile hide behind it.
// 4096 squares in bf16: 1235 TFLOP/s by tiles of 256 (eight wavefronts of 128 x 64), where tiles of 128 reach 0.73 of
// that and of 64 0.55; fp32 143 by 128 (the library's products: 1371 and 150).  LDS has no bank conflicts in any order
// of operands (SQ_LDS_BANK_CONFLICT 0 for each kernel of profiles/layers_counters.txt).
#pragma once

#include "learn.hpp"
#include "parts.hpp"

namespace gnnmb {

// Order of the operands' elements, and the way of a tile into LDS, see above.
enum : int32_t { kForward, kGradX, kGradW };
enum : int32_t { kByPiece, kByWord, kThrough };

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
    int32_t short_segs;                 // segments where fewer than kShortSum of k count; otherwise the last `segs` of them
    int32_t rest;                       // how many of them, the first ones, are of a second plane
    int32_t products;                   // products of the launch (one where it is a gated pair)
    int32_t few;                        // dW of up to kFewRows rows by outer_tile: the columns of one; otherwise 0
    int32_t splits;                     // parts of the summed length, whose sums go to part
    int64_t r_tiles, c_tiles, first_tile;     // set by the launcher
    float *part;                        // [splits][products or pair][rows][ld_part], or NULL: the epilogue follows
    int64_t ld_part;
    Epilogue e;
};

// A rounding of a summed operand to bf16 is as large as the result's own rounding where few terms are
// summed: below this many, the gradients dz are taken in two planes (see dense.hip).
constexpr int64_t kShortSum = 512;

// dW of so few rows is a sum of so many outer products: written by lanes that hold dz, without tiles to fill.
constexpr int kFewRows = 8;

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
            s[i] = z[i] > 0.f ? 1.f : z[i] != z[i] ? z[i] : 0.f;
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
            // where y (1 - y) is 0 the square, which overflows for far z, may be any number
            const float zz = __builtin_fminf(z[i] * z[i], 1e4f);
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

// What is added to V sums: the biases' columns and a row's residual, zeros where there is none.
template <int V>
struct Addends {
    vec<float, V> bias[2], res;
};

template <typename T, int V, bool PAIR>
__device__ __forceinline__ Addends<V> load_addends(const Epilogue &e, int z, int64_t m, int64_t n, int64_t count) {
    Addends<V> x{{vec<float, V>(0.f), vec<float, V>(0.f)}, vec<float, V>(0.f)};
    if (e.bias[z]) x.bias[0] = load_some<T, V>(static_cast<const T *>(e.bias[z]) + n, count);
    if (PAIR && e.bias[1]) x.bias[1] = load_some<T, V>(static_cast<const T *>(e.bias[1]) + n, count);
    if (e.res) x.res = load_some<T, V>(static_cast<const T *>(e.res) + m * e.ld_res + n, count);
    return x;
}

// V values of row m from column n on, `count` of which exist; PAIR: v and u are a gated layer's sums.
template <typename T, int V, bool PAIR>
__device__ __forceinline__ void finish(const Epilogue &e, int z, int64_t m, int64_t n, int64_t count,
                                       vec<float, V> v, vec<float, V> u, const Addends<V> &x) {
    constexpr bool kFast = sizeof(T) == 2;
    v += x.bias[0];
    if (e.pre[z]) store_some<T, V>(static_cast<T *>(e.pre[z]) + m * e.ld_pre + n, count, v);
    v = activate<kFast, V>(e.act, v);
    if (PAIR) {
        u += x.bias[1];
        if (e.pre[1]) store_some<T, V>(static_cast<T *>(e.pre[1]) + m * e.ld_pre + n, count, u);
        v *= u;
    }
    v += x.res;
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
//    other for A, one apart for B; 32 lanes four pieces in a row.  (Lines of eight pieces: 128 bytes.)
//  - Strided fp32: 32 lanes read 128 bytes of one line, the others of the line four below.
template <typename T, bool CONTIGUOUS, bool B, int CPR>
__device__ __forceinline__ int lds_piece(int r, int c) {
    if (CONTIGUOUS) {
        const int low = B ? ((r >> 4) & 1) * 4 + (r & 3) : r & 7;
        return c ^ low ^ ((B ? r >> 2 : r >> 3) & 1);
    }
    if (sizeof(T) == 4) return c ^ ((r >> 2) & 1) * 8;
    if (CPR == 8) return c ^ (B ? (r & 1) | (r & 2) << 1 : (r & 3) * 2);
    return c ^ ((r & 1) * 4 | ((r >> 1) & 1) * 11);
}

// A load from memory into LDS: 16 bytes (or a word) of each lane, from base + offset, to as many bytes times
// the lane from `lds` on (both uniform).  It writes no register; vmcnt counts it, but the compiler does not
// (of the builtin it knows, and waits for all of them before every read of LDS that it cannot tell apart).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"      // that m0 is reserved
template <bool WORD>
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, const void *base) {
    if (WORD)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                     :
                     : "s"(lds), "v"(offset), "s"(base)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(lds), "v"(offset), "s"(base)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

template <int PENDING>
__device__ __forceinline__ void wait_and_meet() {
    static_assert(PENDING < 64, "vmcnt counts 63 loads");
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
template <typename T, bool CONTIGUOUS, bool B, int TILE, int SUB, int THREADS, int LOAD>
struct TileOf {
    static constexpr int kElems = Step<T>::kElems;
    static constexpr int kWide = TILE / SUB;
    static constexpr int kCpr = CONTIGUOUS ? 8 : kWide / kElems;      // pieces per LDS line
    static constexpr int kPieces = TILE * 8 / THREADS;                // pieces per thread
    static constexpr int kBytes = TILE * 128;
    static constexpr int kLinesPerPass = THREADS / kCpr;
    static_assert(kPieces % SUB == 0 && kPieces > 0, "a pass of the threads lies in one stretch");
    static_assert(CONTIGUOUS ? kLinesPerPass % 32 == 0 : kLinesPerPass % 8 == 0, "lds_piece repeats from pass to pass");
    static constexpr bool kWord = LOAD == kByWord;
    static constexpr int kLoads = kWord ? 4 * kPieces : kPieces;      // per thread

    // Line and memory piece of this thread's piece i (within its stretch).
    static __device__ __forceinline__ int line(int i, int t) { return (i % (kPieces / SUB)) * kLinesPerPass + t / kCpr; }
    static __device__ __forceinline__ int piece(int t) {
        return lds_piece<T, CONTIGUOUS, B, kCpr>(t / kCpr, t % kCpr);
    }

    // Byte offsets of the thread's loads from the tile's place in the operand (strided: from the summed index's
    // line; the second stretch has those of the first).  Lines or columns beyond `limit` repeat the last ones; what
    // they give is not stored.
    static constexpr int kOffsets = kWord ? 1 : kPieces / SUB;
    uint32_t offset[kOffsets];
    int64_t first;          // contiguous: first line of the tile
    int64_t limit;
    uint32_t line_bytes;    // kByWord
    uint32_t last;          // kByWord: the last line or element of the tile that exists
    int shift;              // kThrough, strided: elements by which a piece at the lines' end is moved

    __device__ __forceinline__ void init(int64_t first_, int64_t limit_, int64_t ld, int t) {
        first = first_;
        limit = limit_;
        shift = 0;
        if (kWord) {
            line_bytes = static_cast<uint32_t>(ld) * static_cast<uint32_t>(sizeof(T));
            const int64_t left = limit - first - (CONTIGUOUS ? 1 : 4 / static_cast<int>(sizeof(T)));
            last = static_cast<uint32_t>(left < TILE ? left : TILE);
        } else if (CONTIGUOUS) {
#pragma unroll
            for (int i = 0; i < kOffsets; ++i) {
                int64_t r = line(i, t);
                if (first + r >= limit) r = limit - 1 - first;
                offset[i] = static_cast<uint32_t>(r * ld + piece(t) * kElems) * static_cast<uint32_t>(sizeof(T));
            }
        } else {
            int64_t c = first + piece(t) * kElems;
            const int64_t last_piece = limit < kElems ? 0 : limit - kElems;
            if (c > last_piece) {
                if (c < limit) shift = static_cast<int>(c - last_piece);
                c = last_piece;
            }
#pragma unroll
            for (int i = 0; i < kOffsets; ++i)
                offset[i] = static_cast<uint32_t>(c + line(i, t) * ld) * static_cast<uint32_t>(sizeof(T));
        }
    }
    // Where the tile's loads start for summed index k0, and how far it is to the next tile's.
    __device__ __forceinline__ const char *base(const void *p, int64_t ld, int64_t k0) const {
        const int64_t e = CONTIGUOUS ? first * ld + k0 : (kWord ? first : 0) + k0 * ld;
        return static_cast<const char *>(p) + e * static_cast<int64_t>(sizeof(T));
    }
    static __device__ __forceinline__ int64_t advance(int64_t ld) {
        return CONTIGUOUS ? 128 : 128 / static_cast<int>(sizeof(T)) * ld * static_cast<int>(sizeof(T));
    }
    // The thread's offset of load i.
    __device__ __forceinline__ uint32_t at(int i, int t) const {
        if (!kWord) return offset[i % kOffsets];
        constexpr int kLines = THREADS / 4 / kCpr;         // lines per load of all threads
        const int r = (i % (kLoads / SUB)) * kLines + t / 4 / kCpr;
        const uint32_t c = lds_piece<T, CONTIGUOUS, B, kCpr>(r, t / 4 % kCpr) * 16 + t % 4 * 4;     // bytes
        const uint32_t end = CONTIGUOUS ? 0 : last * static_cast<uint32_t>(sizeof(T));
        if (CONTIGUOUS) return (static_cast<uint32_t>(r) < last ? r : last) * line_bytes + c;
        return r * line_bytes + (c < end ? c : end);
    }
    // Bytes of LDS that one load of all threads fills.
    static constexpr int kLoadBytes = THREADS * (kWord ? 4 : 16);

    // Piece i of a tile that the summed length k cuts: what of it exists, shifted to its place, zeros past k.  (Columns
    // past the limit hold anything.)
    __device__ __forceinline__ u4 cut(const void *from, int64_t ld, int i, int64_t k0, int64_t k, int t) const {
        const T *p = static_cast<const T *>(from);
        const int64_t r = CONTIGUOUS ? first + line(i, t) : k0 + line(i, t);
        const int64_t c = (CONTIGUOUS ? k0 : first) + piece(t) * kElems;
        const int64_t lines = CONTIGUOUS ? limit : k, across = CONTIGUOUS ? k : limit;
        p += (r < lines ? r : lines - 1) * ld;
        int64_t over = c + kElems - across;                 // elements that do not exist
        if (over < 0) over = 0;
        u4 v;
        if (across >= kElems) {
            v = __builtin_bit_cast(u4, *reinterpret_cast<const typename loose<T, kElems>::type *>(
                                           p + (over > 0 ? across - kElems : c)));
        } else {
            vec<T, kElems> w(static_cast<T>(0.f));
#pragma unroll
            for (int e = 0; e < kElems; ++e)
                if (e < across) w[e] = p[e];
            v = __builtin_bit_cast(u4, w);
            over -= kElems - across;                        // the piece starts at 0, or past the end
        }
        if (over > 0) v = shifted(v, static_cast<int>(over < kElems ? over : 0));
        if (over >= kElems || (!CONTIGUOUS && r >= k)) v = u4(0);
        return v;
    }
    // A piece that was loaded `by` elements too early, put right.
    static __device__ __forceinline__ u4 shifted(u4 v, int by) {
        const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
        return __builtin_bit_cast(u4, x >> (by * 8 * static_cast<int>(sizeof(T))));
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

// One tile of the product in `lds` (NB buffers of 128 (TR + TC) bytes); q: which tile of which part.
template <typename T, int FORM, int TR, int TC, int WR, int WC, int NB, bool PAIR, int LOAD>
__device__ __forceinline__ void product_tile(const ProductArgs &p, int64_t q, char *lds) {
    constexpr int kThreads = WR * WC * 64;
    constexpr int kBk = 128 / static_cast<int>(sizeof(T));
    constexpr int FR = TR / WR / 32, FC = TC / WC / 32;       // 32 x 32 sums of a wavefront
    static_assert(FR > 0 && FC > 0 && (!PAIR || FC % 2 == 0), "a wavefront holds both sums of a pair");
    constexpr bool kDirect = LOAD != kThrough;
    static_assert(kDirect || NB == 2, "through registers: one tile under way");
    // A wavefront of one 32 x 32 sum in bf16 multiplies 32 cycles a step, where LDS takes over 100 to answer: it has
    // the operands of a whole tile in registers and reads the next one's before it multiplies.  Others have those of a
    // step (fp32, 256 cycles a step: 64 x 64 tiles of 2048 squares 143 us by steps, 150 by whole tiles).
    constexpr bool kWhole = FR * FC == 1 && sizeof(T) == 2;
    typedef TileOf<T, FORM != kGradW, false, TR, 1, kThreads, LOAD> A;
    typedef TileOf<T, FORM == kGradX, true, TC, PAIR ? 2 : 1, kThreads, LOAD> B;
    constexpr int kLoads = A::kLoads + B::kLoads;
    constexpr int kBuffer = A::kBytes + B::kBytes;
    lds_char *const shared = (lds_char *)lds;

    // The tile, and the part of the summed length, of this workgroup.  Workgroups b, b + 8, ... run on one
    // XCD: each XCD takes a stretch of tiles next to each other, whose lines its L2 then holds; the tiles go
    // in columns of eight, so that a stretch is about as high as wide.
    constexpr int64_t kXcds = 8, kHigh = 8;
    const int64_t tiles = p.r_tiles * p.c_tiles;
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
    const int segs = k < kShortSum ? p.short_segs : p.segs, first_seg = p.short_segs - segs;
    const SumPart part = part_of_sum(seg_tiles, segs, p.splits, split);
    const int steps = static_cast<int>(part.steps);
    // Segment and summed index of the next tile to load, and where its loads start (scalars: a look at the
    // arguments for every tile costs 0.1 us of waiting).
    int seg = first_seg + part.seg;
    int64_t k0 = part.tile * kBk;
    const int64_t step_a = A::advance(p.ld_a), step_b = B::advance(p.ld_b);
    const char *from_a, *from_b0, *from_b1;
    const auto place = [&] {
        from_a = ta.base(p.a[seg], p.ld_a, k0);
        from_b0 = tb.base(p.b[z][seg], p.ld_b, k0);
        from_b1 = PAIR ? tb.base(p.b[1][seg], p.ld_b, k0) : from_b0;
    };
    place();

    // A tile narrower than a piece is always taken element by element.
    const bool narrow = !kDirect && ((FORM == kGradW && p.rows < A::kElems) || (FORM != kGradX && p.cols < B::kElems));
    u4 ra[kDirect ? 1 : A::kPieces], rb[kDirect ? 1 : B::kPieces];
    bool staged = false;       // the tile that was last issued waits in ra and rb
    const uint32_t lds0 = static_cast<uint32_t>((uintptr_t)shared);
    auto issue = [&](int buf) {
        if (k0 + kBk <= k && !narrow) {
            if (kDirect) {
                const uint32_t to = lds0 + buf * kBuffer + w * (64 * (A::kWord ? 4 : 16));
#pragma unroll
                for (int i = 0; i < A::kLoads; ++i) load_to_lds<A::kWord>(to + i * A::kLoadBytes, ta.at(i, t), from_a);
#pragma unroll
                for (int i = 0; i < B::kLoads; ++i)
                    load_to_lds<B::kWord>(to + A::kBytes + i * B::kLoadBytes, tb.at(i, t),
                                          PAIR && i >= B::kLoads / 2 ? from_b1 : from_b0);
            } else {
                staged = true;
#pragma unroll
                for (int i = 0; i < A::kPieces; ++i)
                    ra[i] = __builtin_bit_cast(u4, *reinterpret_cast<const typename loose<T, A::kElems>::type *>(from_a + ta.at(i, t)));
#pragma unroll
                for (int i = 0; i < B::kPieces; ++i)
                    rb[i] = __builtin_bit_cast(u4, *reinterpret_cast<const typename loose<T, B::kElems>::type *>(
                                                       (PAIR && i >= B::kPieces / 2 ? from_b1 : from_b0) + tb.at(i, t)));
            }
        } else {
            staged = false;
            const void *pa = p.a[seg], *pb0 = p.b[z][seg], *pb1 = PAIR ? p.b[1][seg] : pb0;
            u4 *to = reinterpret_cast<u4 *>(lds + buf * kBuffer) + t;
            // an operand's pieces under way together (all of both: no registers beside the largest tile's sums)
            u4 va[A::kPieces];
#pragma unroll
            for (int i = 0; i < A::kPieces; ++i) va[i] = ta.cut(pa, p.ld_a, i, k0, k, t);
#pragma unroll
            for (int i = 0; i < A::kPieces; ++i) to[i * kThreads] = va[i];
            __builtin_amdgcn_sched_barrier(0);
            u4 vb[B::kPieces];
#pragma unroll
            for (int i = 0; i < B::kPieces; ++i) vb[i] = tb.cut(PAIR && i >= B::kPieces / 2 ? pb1 : pb0, p.ld_b, i, k0, k, t);
#pragma unroll
            for (int i = 0; i < B::kPieces; ++i) to[A::kBytes / 16 + i * kThreads] = vb[i];
        }
        k0 += kBk;
        from_a += step_a;
        from_b0 += step_b;
        if (PAIR) from_b1 += step_b;
        if (k0 >= k && seg + 1 < p.short_segs) {
            k0 = 0;
            ++seg;
            place();
        }
    };
    // Through registers: the tile that was last issued goes into LDS.
    const bool turned = !kDirect && (p.rows % A::kElems != 0 || p.cols % B::kElems != 0);
    auto commit = [&](int buf) {
        if (kDirect || !staged) return;
        u4 *to = reinterpret_cast<u4 *>(lds + buf * kBuffer) + t;
        if (turned) {
#pragma unroll
            for (int i = 0; i < A::kPieces; ++i) ra[i] = A::shifted(ra[i], ta.shift);
#pragma unroll
            for (int i = 0; i < B::kPieces; ++i) rb[i] = B::shifted(rb[i], tb.shift);
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
    // The products of a second plane come first.  Where one meets an infinity, its sign (or its zero) is not the
    // gradient's: infinity minus infinity would follow.  What of their sums is not finite is dropped, and the first
    // plane gives the infinity or the NaN alone.  drop_at: how many tiles follow the last of them.
    constexpr bool kPlanes = sizeof(T) == 2 && FORM != kForward;
    const int64_t rest64 = (p.rest - first_seg) * seg_tiles - part.first;
    const int drop_at = steps - static_cast<int>(rest64 < 0 ? 0 : rest64 < steps ? rest64 : steps);
    const auto drop = [&](int after) {
        if (!kPlanes || after != drop_at) return;
#pragma unroll
        for (int i = 0; i < FR; ++i)
#pragma unroll
            for (int j = 0; j < FC; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = __builtin_fabsf(acc[i][j][e]) < __builtin_inff() ? acc[i][j][e] : 0.f;
    };
    uint32_t at_a[FR], at_b[FC];
#pragma unroll
    for (int i = 0; i < FR; ++i) at_a[i] = A::read_base(wr * FR + i, lane);
#pragma unroll
    for (int j = 0; j < FC; ++j)
        at_b[j] = A::kBytes + (PAIR ? (j & 1) * (B::kBytes / 2) + B::read_base(wc * (FC / 2) + j / 2, lane)
                                    : B::read_base(wc * FC + j, lane));
    constexpr int kSets = kWhole ? 8 : 2;      // kWhole: 4 set + step; otherwise the parity of the step
    u4 fa[kSets][FR], fb[kSets][FC];
    auto read = [&](int set, int buf, int step, int at) {
        const lds_char *from = shared + buf * kBuffer;
        if (at < FR)
            fa[set][at] = A::read(from, at_a[at], step);
        else
            fb[set][at - FR] = B::read(from, at_b[at - FR], step);
    };
    constexpr int kReads = FR + FC, kProducts = FR * FC;
    // The products of a step, and between them the reads of the next.  (With a tile's loads between them as well, each
    // after one instruction, tiles of 128 and 64 ran 10% slower, and tiles of 256 out of registers.)
    auto multiply = [&](int set, bool next, int buf, int next_step) {
#pragma unroll
        for (int ij = 0; ij < kProducts; ++ij) {
            const int i = ij / FC, j = ij % FC;
            acc[i][j] = Step<T>::mul(fb[set][j], fa[set][i], acc[i][j]);
            if (next) {
#pragma unroll
                for (int r = ij * kReads / kProducts; r < (ij + 1) * kReads / kProducts; ++r)
                    read(next_step & 1, buf, next_step, r);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // The next tile (of `left` that follow the one in hand, in buffer buf) has to be there, and buf has been read.
    auto turn = [&](int buf, int next, int left) {
        commit(next);
        if (NB > 2 && left >= NB - 1)
            wait_and_meet<(NB - 2) * kLoads>();
        else
            wait_and_meet<0>();
        if (left >= (kDirect ? NB : 2)) issue(buf);
    };

    if (steps > 0) {
        if (kDirect) {
#pragma unroll
            for (int j = 0; j < NB - 1; ++j)
                if (j < steps) issue(j);
            if (steps >= NB - 1)
                wait_and_meet<(NB - 2) * kLoads>();
            else
                wait_and_meet<0>();
            if (NB - 1 < steps) issue(NB - 1);
        } else {
            issue(0);
            commit(0);
            wait_and_meet<0>();
            if (steps > 1) issue(1);
        }
        int buf = 0, left = steps - 1;
        if constexpr (kWhole) {
            const auto read_all = [&](int set, int from) {
#pragma unroll
                for (int step = 0; step < 4; ++step)
#pragma unroll
                    for (int r = 0; r < kReads; ++r) read(4 * set + step, from, step, r);
            };
            const auto tile = [&](int set) {
                if (left > 0) {
                    const int next = buf + 1 == NB ? 0 : buf + 1;
                    turn(buf, next, left);
                    read_all(set ^ 1, next);
                    buf = next;
                }
#pragma unroll
                for (int step = 0; step < 4; ++step) multiply(4 * set + step, false, 0, 0);
                drop(left);
            };
            read_all(0, 0);
            while (true) {
                tile(0);
                if (--left < 0) break;
                tile(1);
                if (--left < 0) break;
            }
        } else {
#pragma unroll
            for (int r = 0; r < kReads; ++r) read(0, 0, 0, r);
            // (the second plane's tiles in a loop of their own: with the drop in the loop, sums moved between registers)
            for (int until = kPlanes && drop_at > 0 && drop_at < steps ? drop_at - 1 : 0;; until = 0) {
                for (; left > until; --left) {
                    const int next = buf + 1 == NB ? 0 : buf + 1;
#pragma unroll
                    for (int step = 0; step < 3; ++step) multiply(step & 1, true, buf, step + 1);
                    turn(buf, next, left);
                    multiply(1, true, next, 0);
                    buf = next;
                }
                drop(left + 1);
                if (!kPlanes || left == 0) break;
            }
#pragma unroll
            for (int step = 0; step < 3; ++step) multiply(step & 1, true, buf, step + 1);
            multiply(1, false, 0, 0);
            drop(0);
        }
    }

    // A lane holds row lane % 32 of each 32 x 32 sum, and its columns 16 (lane / 32) + 0..15: place j of them
    // (of the gate's, where there are two).
    constexpr int kPlaces = PAIR ? FC / 2 : FC;
    const auto column = [&](int j) { return c0 + (wc * kPlaces + j) * 32 + (lane >> 5 << 4); };
    const auto row = [&](int i) { return r0 + (wr * FR + i) * 32 + (lane & 31); };
    const auto sum = [&](int i, int j) -> f16x & { return acc[i][PAIR ? 2 * j : j]; };
    const auto other = [&](int i, int j) -> f16x & { return acc[i][PAIR ? 2 * j + 1 : j]; };
    if (p.part) {
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            const int64_t m = row(i);
            if (m >= rows) continue;
            const int64_t at = (split * (PAIR ? 2 : p.products) + z) * p.rows + m;
#pragma unroll
            for (int j = 0; j < kPlaces; ++j) {
                const int64_t n = column(j);
                if (n >= p.cols) continue;
                store_some<float, 16>(p.part + at * p.ld_part + n, p.cols - n, sum(i, j));
                if (PAIR) store_some<float, 16>(p.part + (at + p.rows) * p.ld_part + n, p.cols - n, other(i, j));
            }
        }
        return;
    }
    if (FORM == kForward && sizeof(T) == 2 && FR * FC > 1 && c0 + kPlaces * WC * 32 <= p.cols) {
        // All columns exist, and wavefronts hold many sums: biases are loaded once, a residual's rows a row ahead.
        // (Where each is loaded where it is added, 8192 x 1024 x 4096 bf16 with a bias takes 12% longer and 16384 x 4096 x
        // 4096 with a residual 2%.  fp32 and small tiles lose 5 to 8% to the registers.)
        typedef vec<T, 16> Raw;
        typedef typename loose<T, 16>::type Loose;
        const auto load = [](const void *from, int64_t at) -> Raw { return *reinterpret_cast<const Loose *>(static_cast<const T *>(from) + at); };
        Raw bias[2][kPlaces], res[2][kPlaces];
        const auto load_res = [&](int i) {
            const int64_t m = row(i) < rows ? row(i) : rows - 1;
#pragma unroll
            for (int j = 0; j < kPlaces; ++j) res[i & 1][j] = load(p.e.res, m * p.e.ld_res + column(j));
        };
#pragma unroll
        for (int j = 0; j < kPlaces; ++j) {
            bias[0][j] = bias[1][j] = res[0][j] = res[1][j] = Raw(static_cast<T>(0.f));
            if (p.e.bias[z]) bias[0][j] = load(p.e.bias[z], column(j));
            if (PAIR && p.e.bias[1]) bias[1][j] = load(p.e.bias[1], column(j));
        }
        if (p.e.res) load_res(0);
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            if (p.e.res && i + 1 < FR) load_res(i + 1);
            const int64_t m = row(i);
            if (m >= rows) continue;
#pragma unroll
            for (int j = 0; j < kPlaces; ++j)
                finish<T, 16, PAIR>(p.e, z, m, column(j), 16, sum(i, j), other(i, j),
                                    {{__builtin_convertvector(bias[0][j], f16x), __builtin_convertvector(bias[1][j], f16x)},
                                     __builtin_convertvector(res[i & 1][j], f16x)});
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < FR; ++i) {
        const int64_t m = row(i);
        if (m >= rows) continue;
#pragma unroll
        for (int j = 0; j < kPlaces; ++j) {
            const int64_t n = column(j);
            if (n >= p.cols) continue;
            if (FORM != kForward)
                store_some<T, 16>(static_cast<T *>(p.e.out[z]) + m * p.e.ld_out + n, p.cols - n, sum(i, j));
            else
                finish<T, 16, PAIR>(p.e, z, m, n, p.cols - n, sum(i, j), other(i, j),
                                    load_addends<T, 16, PAIR>(p.e, z, m, n, p.cols - n));
        }
    }
}

// out[c] = the sum of `parts` rows of sums; a workgroup takes 32 columns, a row for every 32 threads at a time.
struct ColumnArgs {
    const float *sums;             // [parts][ld]
    int64_t ld;
    int32_t parts;
    int64_t cols, second;          // out[1] is of the columns from `second` on
    int32_t type;
    void *out[2];                  // may be NULL
    uint32_t blocks;               // workgroups of each of the two (0: nothing to do)
};

template <int THREADS>
__device__ __forceinline__ void column_sums(const ColumnArgs &p, uint32_t block, float *lds) {
    constexpr int kHigh = THREADS / 32;
    const int z = block >= p.blocks ? 1 : 0;
    void *const out = p.out[z];
    if (out == nullptr) return;      // whole workgroup
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t c = (block - z * p.blocks) * 32ll + x;
    float s = 0.f;
    if (c < p.cols) {
        const float *from = p.sums + z * p.second + c;
#pragma unroll 8
        for (int i = y; i < p.parts; i += kHigh) s += from[i * p.ld];
    }
    lds[y * 33 + x] = s;
    __syncthreads();
    if (y == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < kHigh; ++i) s += lds[i * 33 + x];
        if (p.type == GNN_BF16)
            static_cast<bf16 *>(out)[c] = static_cast<bf16>(s);
        else
            static_cast<float *>(out)[c] = s;
    }
}

// dW = x^T dz for up to kFewRows rows.  A lane holds its 16 bytes' columns of every row of dz (both planes of it,
// added), a wavefront writes kOuterHigh lines of dW; x comes from LDS.  What bounds it is the writing.  All gradients
// of 4 rows of 4096 x 4096 bf16 with gelu take 28 us, 52 where tiles of the matrix units are filled, cut and emptied
// for dW; of one row of 7168 x 6464 fp32 88 and 168 (70 at 5.4 TB/s).
constexpr int kOuterHigh = 16;

template <typename T>
constexpr int kOuterWide = 64 * 16 / static_cast<int>(sizeof(T));

template <typename T, int THREADS>
__device__ __forceinline__ void outer_tile(const ProductArgs &p, int64_t q, float *lds) {
    constexpr int V = 16 / static_cast<int>(sizeof(T)), kHigh = kOuterHigh * THREADS / 64;
    typedef vec<float, V> Wide;
    const int64_t tiles = p.r_tiles * p.c_tiles, z = q / tiles;
    q -= z * tiles;
    const int64_t tr = q / p.c_tiles, r0 = tr * kHigh, n = load_count(p.d_n, p.k);
    const int t = threadIdx.x, lane = lane_id(), w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t at = (q - tr * p.c_tiles) * kOuterWide<T> + lane * V;
    const int64_t c = at < p.cols - V ? at : p.cols - V;      // the last lanes' columns overlap, with the same results
    for (int e = t; e < kHigh * kFewRows; e += THREADS) {
        const int i = e % kHigh, row = e / kHigh;
        const bool there = row < n && r0 + i < p.rows;
        lds[i * kFewRows + row] = there ? static_cast<float>(static_cast<const T *>(p.a[0])[row * p.ld_a + r0 + i]) : 0.f;
    }
    Wide dz[kFewRows];
#pragma unroll
    for (int row = 0; row < kFewRows; ++row) {
        dz[row] = Wide(0.f);
        if (row < n) {
            dz[row] = load_f32<T, V>(static_cast<const T *>(p.b[z][0]) + row * p.ld_b + c);
            if (p.short_segs > 1) dz[row] += load_f32<T, V>(static_cast<const T *>(p.b[z][1]) + row * p.ld_b + c);
        }
    }
    __syncthreads();
    T *const out = static_cast<T *>(p.e.out[z]) + c;
#pragma unroll 4
    for (int i = 0; i < kOuterHigh; ++i) {
        const int64_t r = r0 + w * kOuterHigh + i;
        if (r >= p.rows) break;
        const float *x = lds + (w * kOuterHigh + i) * kFewRows;
        Wide v = x[0] * dz[0];
#pragma unroll
        for (int row = 1; row < kFewRows; ++row) v += x[row] * dz[row];
        store_f32<T, V>(out + r * p.e.ld_out, v);
    }
}

// Wavefronts, buffers of LDS (by the type's bytes) and wavefronts a SIMD of each tile shape.
struct Tile256 {          // bf16 only, by pieces only
    static constexpr int kRows = 256, kCols = 256, kWr = 2, kWc = 4;
    static constexpr int buffers(int, int) { return 2; }
    static constexpr int waves(int, int) { return 2; }
};
struct Tile128 {          // bf16 straight into LDS: one workgroup a compute unit (large bf16 products take Tile256);
                          // through registers two (gradients of 4096 x 1031 x 4097 186 us, 241 by one)
    static constexpr int kRows = 128, kCols = 128, kWr = 2, kWc = 2;
    static constexpr int buffers(int size, int load) { return size == 4 || load == kThrough ? 2 : load == kByWord ? 3 : 4; }
    static constexpr int waves(int size, int load) { return size == 2 && load != kThrough ? 1 : 2; }
};
struct Tile64 {
    static constexpr int kRows = 64, kCols = 64, kWr = 2, kWc = 2;
    static constexpr int buffers(int, int load) { return load == kThrough ? 2 : 4; }
    static constexpr int waves(int, int) { return 2; }
};
struct Tile32 {           // few rows
    static constexpr int kRows = 32, kCols = 128, kWr = 1, kWc = 4;
    static constexpr int buffers(int, int load) { return load == kThrough ? 2 : 4; }
    static constexpr int waves(int, int) { return 2; }
};

template <typename T, typename TILE, bool PAIR, int LOAD>
__global__ __launch_bounds__(TILE::kWr * TILE::kWc * 64, TILE::waves(sizeof(T), LOAD)) void k_product(ProductArgs p) {
    constexpr int NB = TILE::buffers(sizeof(T), LOAD);
    __shared__ __align__(1024) char lds[NB * (TILE::kRows + TILE::kCols) * 128];
    product_tile<T, kForward, TILE::kRows, TILE::kCols, TILE::kWr, TILE::kWc, NB, PAIR, LOAD>(p, p.first_tile + blockIdx.x, lds);
}

// Both gradients of a layer, and the sums of the bias's: w_tiles workgroups of dW, x_tiles of dx (those whose summed
// length is longer come first, so that none of them is left at the end), and the last ones add columns.
template <typename T, typename TILE, int LOAD>
__global__ __launch_bounds__(TILE::kWr * TILE::kWc * 64, TILE::waves(sizeof(T), LOAD)) void k_gradients(
    ProductArgs w, ProductArgs x, ColumnArgs c, int64_t w_tiles, int64_t x_tiles, bool x_first) {
    constexpr int NB = TILE::buffers(sizeof(T), LOAD);
    __shared__ __align__(1024) char lds[NB * (TILE::kRows + TILE::kCols) * 128];
    const int64_t q = w.first_tile + blockIdx.x, all = w_tiles + x_tiles;
    const int64_t qw = x_first ? q - x_tiles : q, qx = x_first ? q : q - w_tiles;
    if (q >= all)
        column_sums<TILE::kWr * TILE::kWc * 64>(c, static_cast<uint32_t>(q - all), reinterpret_cast<float *>(lds));
    else if ((x_first ? qw >= 0 : qx < 0) && w.few)
        outer_tile<T, TILE::kWr * TILE::kWc * 64>(w, qw, reinterpret_cast<float *>(lds));
    else if (x_first ? qw >= 0 : qx < 0)
        product_tile<T, kGradW, TILE::kRows, TILE::kCols, TILE::kWr, TILE::kWc, NB, false, LOAD>(w, qw, lds);
    else
        product_tile<T, kGradX, TILE::kRows, TILE::kCols, TILE::kWr, TILE::kWc, NB, false, LOAD>(x, qx, lds);
}

// ---- launching --------------------------------------------------------------------------------------

enum : int32_t { kTile256, kTile128, kTile64, kTile32 };

inline int tile_rows(int tile) { return tile == kTile256 ? 256 : tile == kTile128 ? 128 : tile == kTile64 ? 64 : 32; }
inline int tile_cols(int tile, bool pair) {
    return (tile == kTile256 ? 256 : tile == kTile64 ? 64 : 128) / (pair ? 2 : 1);
}

// pair: the two products' sums meet in one workgroup (kTile256 and kTile128); load: kByPiece, kByWord or kThrough.
hipError_t launch_product_bf16(ProductArgs a, int tile, bool pair, int load, hipStream_t s);
hipError_t launch_product_f32(ProductArgs a, int tile, bool pair, int load, hipStream_t s);
// Either of w and x may have no products.
hipError_t launch_gradients_bf16(ProductArgs w, ProductArgs x, const ColumnArgs &c, int tile, int load, hipStream_t s);
hipError_t launch_gradients_f32(ProductArgs w, ProductArgs x, const ColumnArgs &c, int tile, int load, hipStream_t s);

inline int64_t set_tiles(ProductArgs &a, int tile, bool pair) {
    if (a.few) {
        const int64_t high = kOuterHigh * (tile == kTile256 ? 8 : 4);
        a.r_tiles = (a.rows + high - 1) / high;
        a.c_tiles = (a.cols + a.few - 1) / a.few;
        return a.r_tiles * a.c_tiles * a.products;
    }
    a.r_tiles = (a.rows + tile_rows(tile) - 1) / tile_rows(tile);
    a.c_tiles = (a.cols + tile_cols(tile, pair) - 1) / tile_cols(tile, pair);
    return a.r_tiles * a.c_tiles * a.products * a.splits;
}

template <typename T, typename TILE, bool PAIR, int LOAD>
hipError_t launch_tiles(ProductArgs &a, int64_t tiles, hipStream_t s) {
    constexpr int kThreads = TILE::kWr * TILE::kWc * 64;
    return launch_pieces(tiles, kThreads, [&](int64_t first, unsigned blocks) {
        a.first_tile = first;
        k_product<T, TILE, PAIR, LOAD><<<blocks, kThreads, 0, s>>>(a);
    });
}

template <typename T, typename TILE, bool PAIR>
hipError_t launch_by(ProductArgs &a, int load, int64_t tiles, hipStream_t s) {
    if (load == kByPiece) return launch_tiles<T, TILE, PAIR, kByPiece>(a, tiles, s);
    if (sizeof(T) == 4 || load == kByWord) return launch_tiles<T, TILE, PAIR, kByWord>(a, tiles, s);
    if constexpr (sizeof(T) == 2) return launch_tiles<T, TILE, PAIR, kThrough>(a, tiles, s);
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_product(ProductArgs a, int tile, bool pair, int load, hipStream_t s) {
    const int64_t tiles = set_tiles(a, tile, pair);
    if constexpr (sizeof(T) == 2) {
        if (tile == kTile256)
            return pair ? launch_tiles<T, Tile256, true, kByPiece>(a, tiles, s) : launch_tiles<T, Tile256, false, kByPiece>(a, tiles, s);
    }
    if (tile == kTile32) return launch_by<T, Tile32, false>(a, load, tiles, s);
    if (tile == kTile64) return launch_by<T, Tile64, false>(a, load, tiles, s);
    return pair ? launch_by<T, Tile128, true>(a, load, tiles, s) : launch_by<T, Tile128, false>(a, load, tiles, s);
}

template <typename T, typename TILE, int LOAD>
hipError_t launch_both(ProductArgs &w, ProductArgs &x, const ColumnArgs &c, int64_t w_tiles, int64_t x_tiles, hipStream_t s) {
    constexpr int kThreads = TILE::kWr * TILE::kWc * 64;
    const bool x_first = w.few || x.k * x.segs * w.splits > w.k * w.segs * x.splits;
    return launch_pieces(w_tiles + x_tiles + 2 * c.blocks, kThreads, [&](int64_t first, unsigned blocks) {
        w.first_tile = first;
        k_gradients<T, TILE, LOAD><<<blocks, kThreads, 0, s>>>(w, x, c, w_tiles, x_tiles, x_first);
    });
}

template <typename T, typename TILE>
hipError_t launch_both_by(ProductArgs &w, ProductArgs &x, const ColumnArgs &c, int load, int64_t w_tiles, int64_t x_tiles,
                          hipStream_t s) {
    if (load == kByPiece) return launch_both<T, TILE, kByPiece>(w, x, c, w_tiles, x_tiles, s);
    if (sizeof(T) == 4 || load == kByWord) return launch_both<T, TILE, kByWord>(w, x, c, w_tiles, x_tiles, s);
    if constexpr (sizeof(T) == 2) return launch_both<T, TILE, kThrough>(w, x, c, w_tiles, x_tiles, s);
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_gradients(ProductArgs w, ProductArgs x, const ColumnArgs &c, int tile, int load, hipStream_t s) {
    const int64_t w_tiles = set_tiles(w, tile, false), x_tiles = set_tiles(x, tile, false);
    if constexpr (sizeof(T) == 2) {
        if (tile == kTile256) return launch_both<T, Tile256, kByPiece>(w, x, c, w_tiles, x_tiles, s);
    }
    if (tile == kTile64) return launch_both_by<T, Tile64>(w, x, c, load, w_tiles, x_tiles, s);
    return launch_both_by<T, Tile128>(w, x, c, load, w_tiles, x_tiles, s);
}

}  // namespace gnnmb
