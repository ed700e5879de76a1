// Orthogonalising a weight matrix's update by Newton-Schulz products (the step of the Muon optimiser).
//
// With X = G / (|G|_F + eps), every step applies the odd polynomial p(s) = a s + b s^3 + c s^5 to the
// singular values of X, by products alone:
//   A = X X^T,   Q = a I + b A + c A^2,   X <- Q X,
// X taken wide (s rows, l >= s columns), so that A and Q are s x s.  A and Q are symmetric: one
// triangle of their tiles is computed, and each tile is stored a second time, mirrored.
//
// Numbers.  The products run on the 16-bit matrix instructions with fp32 accumulation.  X, A and Q
// are stored in fp16, times 2^12: the singular values stay below 3 (newton_in_range), so that
// every entry fits, and entries down to 2^-26 keep fp16's 11 bits.  A bf16 update takes one fp16 plane, eight
// times the precision of its own entries (directions below 2^-9 of the strongest are as much its own
// rounding as the update), and what the plane leaves of the diagonals of A and Q, in fp32.  Those are
// often alike, and one rounding common to all of them scales the whole result, by up to half a step of
// bf16 (400 x 4000 orthonormal rows: 1.8e-3 of it; the diagonals' rest brings the error from 1.9 times the
// result's own rounding to 1.05, and is 1.14 at most over Gaussian, orthonormal and low-rank updates of
// 3 to 700 rows); the other entries' roundings are of either sign.  The fp32 update takes two planes,
// x = hi + lo (22 bits), and three matrix products, hi hi + hi lo + lo hi (all four for small matrices);
// the dropped product is below 2^-22 of a term.  The first X is G times a power of two, so
// nothing is rounded that need not be, and the rest of 1 / (|G|_F + eps) multiplies the first A and the
// first Q X.
//
// Layout.  The matrix instructions want both operands with the summed index contiguous: X for A, the
// symmetric A for A^2, and, since (Q X)^T = X^T Q, X^T and Q for the last product, which therefore
// stores X and X^T.  The planes are padded with zeros to multiples of 64, and zeros stay zeros; a tile
// that reaches beyond them repeats their last row and stores nothing there.
//
// What bounds it.  Large squares: LDS reads and the tiles' way into it next to the matrix units: five
// steps of 4096 x 4096 bf16 in 1.62 ms, 850 TFLOP/s of the needed operations (a library product reaches
// 1050 to 1150 at this size).  Two planes: 2 x 2571 x 1030 fp32 710 us, three products for one.  Small ones:
// the chain of three products a step; 256 x 256 fp32 takes 119 us in 17 launches of about 7 us each, of
// which 2.6 are the launch's own, 0.7 the first load and 0.9 the stores.
#include <math.h>

#include "learn.hpp"

namespace gnnmb {

namespace {

typedef _Float16 f16;
typedef vec<f16, 8> h8;
typedef vec<float, 16> f16x;

constexpr float kUp = 4096.f;                 // the stored planes' factor, 2^12
constexpr float kDown = 1.f / 4096.f;

// Where the tile's 16-byte piece c of row r lies in LDS, in pieces: a row's pieces are permuted by the
// row, so that the 32 rows which one operand read touches at the same c spread over the banks.
template <int CPR>
__device__ __forceinline__ int piece(int r, int c) {
    return r * CPR + (c ^ ((CPR == 8 ? r : r >> 1) & (CPR - 1)));
}

enum : int32_t { kGram, kPoly, kApply, kLast };

struct ProductArgs {
    const f16 *a, *b;            // [rows, ld] planes, summed index contiguous
    int64_t ld_a, ld_b, plane_a, plane_b, batch_a, batch_b;
    f16 *c, *t;                  // the product, and its transpose (symmetric: the mirrored tiles)
    int64_t ld_c, ld_t, plane_c, plane_t, batch_c, batch_t;
    int64_t k;                   // summed length, a multiple of 64
    int32_t rows_a, rows_b;      // padded rows of the operands: multiples of 64
    int32_t m_tiles, n_tiles;
    int32_t what;
    float ca, cb, cc;            // kPoly
    const float *first;          // [batch] factor of X in the first step, NULL: 1
    // one plane: [batch][ld_rest] what the planes leave of the diagonals (times 2^12): of A, written by
    // kGram and read by kPoly, and of Q, written by kPoly and read by the last product
    float *rest_a, *rest_q;
    int64_t ld_rest;
    // kLast
    void *out;
    int64_t ld_out, batch_out;
    int64_t m, n;                // rows and columns of the product that exist
    int32_t out_rows;            // 1: out[m][n], 0: out[n][m]
    float scale;
};

template <int PL>
struct PolyOf {
    typedef float type;
};
// The terms of a + b A + c A^2 cancel to a fraction of their size, so for fp32 updates they are added
// in 64 bits (an s x s epilogue: no time that shows).
template <>
struct PolyOf<2> {
    typedef double type;
};

constexpr int kThreads = 256;      // four wavefronts, two by two quarters of a tile
// Tiles on their way (even: LDS has two halves): as many as leave two workgroups per compute unit at
// TILE = 128 their registers.
template <int TILE>
constexpr int depth() {
    return TILE == 128 ? 2 : 4;
}

// One TILE x TILE tile of the product.  A wavefront's quarter is TM x TM matrix instructions of 32 x 32 a
// summed sixteen; an operand piece that it reads from LDS is used TM times, so LDS keeps up from TM = 3
// on (at TM = 2 it delivers just what the matrix units take).  The operands of the next sixteen are
// read while those of the last multiply.  A tile of the planes takes longer to arrive than a turn's
// products (some 2000 cycles against 512 at TILE = 128), so kDepth tiles are on their way at once, in
// register sets of their own; the next one is put into the other half of LDS before a turn's last
// products.
template <int TILE, int PL, typename TO>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void k_newton_product(ProductArgs p) {
    constexpr int BK = PL == 1 ? 64 : 32;
    constexpr int CPR = BK / 8;                     // 16-byte pieces per row
    constexpr int KK = BK / 16;
    constexpr int TM = TILE / 64;
    constexpr int kDepth = depth<TILE>();
    constexpr int L = TILE * CPR / kThreads;        // pieces per thread, operand and plane
    // Small matrices are not bound by the products, and their sums are too short for the dropped one
    // to average out (1.2e-6 of a 5 x 1 update's norm without it, 1e-7 with it).
    constexpr bool kAllFour = TILE == 64;
    typedef typename PolyOf<PL>::type Poly;
    constexpr int kPlane = 2 * TILE * CPR;          // an A and a B tile
    __shared__ h8 lds[2][PL * kPlane];
    const bool symmetric = p.what == kGram || p.what == kPoly;
    // Workgroups b, b + 8, ... run on one XCD: each XCD takes a stretch of tiles next to each other, whose
    // rows its L2 then holds.
    constexpr unsigned kXcds = 8;
    const unsigned whole = gridDim.x / kXcds * kXcds;
    const int q0 = static_cast<int>(blockIdx.x < whole
                                        ? blockIdx.x % kXcds * (whole / kXcds) + blockIdx.x / kXcds
                                        : blockIdx.x);
    int tm, tn;
    if (symmetric) {
        tm = static_cast<int>((sqrtf(8.f * q0 + 1.f) - 1.f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= q0) ++tm;
        while (tm * (tm + 1) / 2 > q0) --tm;
        tn = q0 - tm * (tm + 1) / 2;
    } else {
        // columns of four tiles, so that a stretch is about as wide as high
        const int per = 4 * p.n_tiles, g = q0 / per, in = q0 - g * per;
        const int high = p.m_tiles - 4 * g < 4 ? p.m_tiles - 4 * g : 4;
        tn = in / high;
        tm = 4 * g + in - tn * high;
    }
    const int64_t z = blockIdx.y;
    const int t = threadIdx.x, lane = lane_id(), w = t >> 6;
    const int wm = w >> 1, wn = w & 1;
    const f16 *ga = p.a + z * p.batch_a;
    const f16 *gb = p.b + z * p.batch_b;
    // this thread's pieces: row and distance from the planes' start
    uint32_t oa[L], ob[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int e = i * kThreads + t, r = e / CPR, c = e % CPR;
        const int ra = tm * TILE + r, rb = tn * TILE + r;
        oa[i] = static_cast<uint32_t>(ra < p.rows_a ? ra : p.rows_a - 1) * static_cast<uint32_t>(p.ld_a) + c * 8;
        ob[i] = static_cast<uint32_t>(rb < p.rows_b ? rb : p.rows_b - 1) * static_cast<uint32_t>(p.ld_b) + c * 8;
    }
    h8 ra[kDepth][PL][L], rb[kDepth][PL][L];
    const int steps = static_cast<int>(p.k / BK);
    // The pieces of a turn: plane, operand, and which of the thread's.  (Past the end the last tile is
    // loaded again: no branch, so that the waits count the loads exactly.)
    constexpr int kPieces = PL * 2 * L;
    auto load = [&](int set, int s, int at) {
        const int64_t k0 = static_cast<int64_t>(s < steps ? s : steps - 1) * BK;
        const int q = at / (2 * L), i = at % L;
        if (at % (2 * L) < L)
            ra[set][q][i] = *reinterpret_cast<const h8 *>(ga + q * p.plane_a + k0 + oa[i]);
        else
            rb[set][q][i] = *reinterpret_cast<const h8 *>(gb + q * p.plane_b + k0 + ob[i]);
    };
    auto store = [&](int set, int buf, int at) {
        const int q = at / (2 * L), i = at % L, e = i * kThreads + t;
        h8 *to = &lds[buf][q * kPlane + piece<CPR>(e / CPR, e % CPR)];
        if (at % (2 * L) < L)
            *to = ra[set][q][i];
        else
            to[TILE * CPR] = rb[set][q][i];
    };
    // Two planes: what hi lo, lo hi and lo lo add is some 2^-12 of the sum, and is summed apart, so that the
    // sum itself is rounded once a product of sixteen and not three times (long sums: 4 x 3290 x 138 fp32 is
    // off by 1.8e-6 so, 3.0e-6 otherwise).
    f16x acc[TM][TM], small[PL == 2 ? TM : 1][PL == 2 ? TM : 1];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            acc[i][j] = f16x(0.f);
            if (PL == 2) small[i][j] = f16x(0.f);
        }

    const int row = lane & 31, half = lane >> 5;
    h8 a[2][PL][TM], b[2][PL][TM];
    constexpr int kReads = PL * 2 * TM;
    auto read = [&](int buf, int kk, int at) {
        const int q = at / (2 * TM), i = at % TM;
        const h8 *pl = &lds[buf][q * kPlane];
        if (at % (2 * TM) < TM)
            a[kk & 1][q][i] = pl[piece<CPR>((wm * TM + i) * 32 + row, kk * 2 + half)];
        else
            b[kk & 1][q][i] = pl[TILE * CPR + piece<CPR>((wn * TM + i) * 32 + row, kk * 2 + half)];
    };
    // Tile s, from LDS half s % 2; u = s % kDepth, whose register set is free.  Between any two products
    // comes a share of the turn's other work (the next operands, the loads kDepth tiles ahead, the next
    // tile's way into LDS): in a row, with no product under way, the loads alone take 670 cycles of a
    // turn and the stores 600 beside the 1152 of its products (TILE = 192).
    auto turn = [&](int u, int s) {
        const int buf = u & 1;
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(buf, 0, r);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const auto &x = a[kk & 1];
            const auto &y = b[kk & 1];
#pragma unroll
            for (int ij = 0; ij < TM * TM; ++ij) {
                const int i = ij / TM, j = ij % TM;
                if (PL == 2) {
                    if (kAllFour)
                        small[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[PL - 1][i], y[PL - 1][j], small[i][j], 0, 0, 0);
                    small[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[0][i], y[PL - 1][j], small[i][j], 0, 0, 0);
                    small[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[PL - 1][i], y[0][j], small[i][j], 0, 0, 0);
                }
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[0][i], y[0][j], acc[i][j], 0, 0, 0);
                if (kk + 1 < KK) {
#pragma unroll
                    for (int r = ij * kReads / (TM * TM); r < (ij + 1) * kReads / (TM * TM); ++r) read(buf, kk + 1, r);
                }
                constexpr int kSlots = KK * TM * TM;
                const int slot = kk * TM * TM + ij;
#pragma unroll
                for (int r = slot * kPieces / kSlots; r < (slot + 1) * kPieces / kSlots; ++r) {
                    load(u, s + kDepth, r);
                    store((u + 1) % kDepth, buf ^ 1, r);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
    };
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
#pragma unroll
        for (int r = 0; r < kPieces; ++r) load(u, u, r);
        __builtin_amdgcn_sched_barrier(0);      // in this order: the first tile is waited for alone
    }
#pragma unroll
    for (int r = 0; r < kPieces; ++r) store(0, 0, r);
    __syncthreads();
    int s = 0;
    for (; s + kDepth <= steps; s += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) turn(u, s + u);
    }
#pragma unroll
    for (int u = 0; u < kDepth - 1; ++u)
        if (s + u < steps) turn(u, s + u);
    if (PL == 2) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] += small[i][j];
    }

    // A lane holds column lane % 32 and rows 8 g + 4 (lane / 32) + 0..3 of each 32 x 32 accumulator:
    // every(f) calls f(row, column, the four values) for what exists of the padded product.  A padded
    // plane has at most 2^30 elements.
    const auto every = [&](auto f) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int n = tn * TILE + (wn * TM + j) * 32 + row;
                const int m0 = tm * TILE + (wm * TM + i) * 32 + 4 * half;
                // a 32 x 32 accumulator exists or not as a whole
                if (n >= p.rows_b || m0 >= p.rows_a) continue;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    f(m0 + 8 * g, n,
                      vec<float, 4>{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
            }
    };
    const float first = p.first ? p.first[z] : 1.f;
    float *rest_a = nullptr, *rest_q = nullptr;
    if constexpr (PL == 1) {
        rest_a = p.rest_a + z * p.ld_rest;
        rest_q = p.rest_q + z * p.ld_rest;
        if (!symmetric) {
            // X^T Q (a holds X^T): what Q's plane leaves of its diagonal, times X itself.  All loads before any
            // store.
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int n = tn * TILE + (wn * TM + j) * 32 + row;
                if (n >= p.rows_b) continue;
                const float rest = rest_q[n];
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int m0 = tm * TILE + (wm * TM + i) * 32 + 4 * half;
                    if (m0 >= p.rows_a) continue;
                    const f16 *x = ga + m0 * p.ld_a + n;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[i][j][e] += rest * static_cast<float>(x[(8 * (e >> 2) + (e & 3)) * p.ld_a]);
                }
            }
        }
    }
    if (p.what == kLast) {
        const float factor = kDown * kDown * first * p.scale;
        TO *out = static_cast<TO *>(p.out) + z * p.batch_out;
        const int rows = static_cast<int>(p.m), cols = static_cast<int>(p.n);
        every([&](int m, int n, vec<float, 4> v) {
            v *= factor;
            if (n >= cols) return;
            if (!p.out_rows && m + 4 <= rows) {
                store_f32<TO, 4>(out + n * p.ld_out + m, v);
                return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < rows) out[p.out_rows ? (m + e) * p.ld_out + n : n * p.ld_out + m + e] = static_cast<TO>(v[e]);
        });
        return;
    }
    const bool mirror = !symmetric || tm != tn;
    char *const pc = reinterpret_cast<char *>(p.c + z * p.batch_c);
    char *const pt = reinterpret_cast<char *>(p.t + z * p.batch_t);
    const uint32_t ld_c = static_cast<uint32_t>(p.ld_c), ld_t = static_cast<uint32_t>(p.ld_t);
    const auto keep = [&](int m, int n, vec<float, 4> v, float *rest) {
        const uint32_t oc = 2 * (m * ld_c + n), ot = 2 * (n * ld_t + m);
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const vec<f16, 4> x = __builtin_convertvector(v, vec<f16, 4>);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f16 *>(pc + 2 * q * p.plane_c + (oc + 2 * e * ld_c)) = x[e];
            if (mirror) *reinterpret_cast<vec<f16, 4> *>(pt + 2 * q * p.plane_t + ot) = x;
            v -= __builtin_convertvector(x, vec<float, 4>);
        }
        if (PL == 1 && rest != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e == n) rest[n] = v[e];
        }
    };
    if (p.what == kPoly) {
        // the product's operand is A itself, A[n][m..] = A[m..][n]
        const char *const old = reinterpret_cast<const char *>(p.a + z * p.batch_a);
        const uint32_t ld_a = static_cast<uint32_t>(p.ld_a);
        every([&](int m, int n, vec<float, 4> v) {
            if constexpr (PL == 1) {
                // (A + R)^2 = A^2 + R A + A R + R^2, R being the diagonal's rest
                const vec<f16, 4> x = *reinterpret_cast<const vec<f16, 4> *>(old + 2 * (n * ld_a + m));
                const float rn = rest_a[n];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float rm = rest_a[m + e], y = static_cast<float>(x[e]);
                    v[e] += (rm + rn) * y;
                    if (m + e == n) v[e] += rn * rn;
                    v[e] = v[e] * (kDown * p.cc) + p.cb * y;
                    if (m + e == n) v[e] += p.cb * rn + p.ca * kUp;
                }
                keep(m, n, v, rest_q);
                return;
            }
            vec<Poly, 4> u = __builtin_convertvector(v, vec<Poly, 4>) * static_cast<Poly>(kDown * p.cc);
#pragma unroll
            for (int q = 0; q < PL; ++q) {
                const vec<f16, 4> x =
                    *reinterpret_cast<const vec<f16, 4> *>(old + 2 * q * p.plane_a + 2 * (n * ld_a + m));
                u += static_cast<Poly>(p.cb) * __builtin_convertvector(x, vec<Poly, 4>);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e == n) u[e] += static_cast<Poly>(p.ca * kUp);
            keep(m, n, __builtin_convertvector(u, vec<float, 4>), nullptr);
        });
    } else {
        const float factor = kDown * first * (p.what == kGram ? first : 1.f);
        float *const rest = p.what == kGram ? rest_a : nullptr;
        every([&](int m, int n, vec<float, 4> v) { keep(m, n, v * factor, rest); });
    }
}

// ---- the norm and the first X ---------------------------------------------------------------------

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 256;     // most partial sums per matrix: one per thread of the reader

struct PrepArgs {
    const void *g;
    int64_t rows, cols, ld, batch_g;
    double *partial;        // [batch, blocks] sums of squares
    int32_t blocks;
    float eps;
    float *first;           // [batch]
    f16 *same, *turned;     // G's orientation, and transposed; padded
    int64_t ld_same, ld_turned, plane, batch;   // elements
};

// Squares are summed in 64 bits, which neither overflow nor vanish for any fp32 update.
template <typename TI>
__global__ __launch_bounds__(kNormThreads) void k_norm_squares(PrepArgs p) {
    __shared__ double sm[kNormThreads / 64];
    const TI *g = static_cast<const TI *>(p.g) + blockIdx.y * p.batch_g;
    const int w = threadIdx.x >> 6;
    double sum = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + w; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * 4)
#pragma unroll 8
        for (int64_t c = lane_id(); c < p.cols; c += 64) {
            const double x = static_cast<float>(g[r * p.ld + c]);
            sum += x * x;
        }
    sum = wave_sum(sum);
    if (lane_id() == 0) sm[w] = sum;
    __syncthreads();
    if (threadIdx.x == 0) p.partial[blockIdx.y * p.blocks + blockIdx.x] = (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

template <typename TI, int PL>
__global__ __launch_bounds__(kNormThreads) void k_first_planes(PrepArgs p) {
    __shared__ double sm[kNormThreads / 64];
    __shared__ f16 tile[PL][64][66];
    const int t = threadIdx.x, w = t >> 6;
    const int64_t z = blockIdx.z;
    // the tile's values, every load made, of a place that exists, while the norm is put together
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
    const TI *g = static_cast<const TI *>(p.g) + z * p.batch_g;
    const int64_t col = c0 + (t & 63) < p.cols ? c0 + (t & 63) : p.cols - 1;
    TI raw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + w * 16 + i;
        raw[i] = g[(r < p.rows ? r : p.rows - 1) * p.ld + col];
    }
    const double s = wave_sum(t < p.blocks ? p.partial[z * p.blocks + t] : 0.0);
    if (lane_id() == 0) sm[w] = s;
    __syncthreads();
    const double norm = sqrt((sm[0] + sm[1]) + (sm[2] + sm[3]));
    int e = 0;
    if (norm > 0 && norm <= 1.7e308) frexp(norm, &e);     // norm 2^-e in [0.5, 1)
    if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) {
        // the rest of the division, exactly 0 for a zero update and NaN where G is not finite
        double rest = norm > 0 ? 1.0 / ldexp(norm + static_cast<double>(p.eps), -e) : 0.0;
        if (!(norm <= 1.7e308)) rest = __builtin_nan("");
        p.first[z] = static_cast<float>(rest);
    }
    const int c = t & 63;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = w * 16 + i;
        float v = 0.f;
        if (r0 + r < p.rows && c0 + c < p.cols) v = ldexpf(static_cast<float>(raw[i]), 12 - e);
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const f16 x = static_cast<f16>(v);
            p.same[z * p.batch + q * p.plane + (r0 + r) * p.ld_same + c0 + c] = x;
            tile[q][c][r] = x;
            v -= static_cast<float>(x);
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < PL; ++q)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = w * 16 + i;
            p.turned[z * p.batch + q * p.plane + (c0 + r) * p.ld_turned + r0 + c] = tile[q][r][c];
        }
}

// ---- host -------------------------------------------------------------------------------------------

struct NewtonSpace {
    f16 *x, *xt[2], *a, *q;
    float *first, *rest_a, *rest_q;      // (rests: [batch][s])
    double *partial;
    int64_t s, l;           // padded
    int64_t plane_x, plane_a;
    int32_t planes;
    size_t bytes;
};

// The tile edge of a product: the one whose tiles the compute units are through with first.  A tile's
// time is its area over the rate at this edge, for a compute unit's only tile and for several.  Rates
// relative to an edge of 192, from five steps on bf16 squares with one edge throughout: 4096 (several
// tiles a unit) takes 1.65 ms by 192, 1.97 by 128, 2.89 by 64; 1024 (at most one) 364 us by 192, 228 by 128,
// 145 by 64; 2048 530, 376 and 455 us.  Two planes at 192 exceed the registers.
int32_t tile_for(int64_t rows_a, int64_t rows_b, int64_t batch, bool symmetric, int planes) {
    const int32_t edge[3] = {192, 128, 64};
    const double many[3] = {1.0, 0.85, 0.57}, alone[3] = {1.0, 0.9, 0.57};
    int32_t best = 64;
    double least = 0;
    for (int i = planes - 1; i < 3; ++i) {
        const int64_t m = (rows_a + edge[i] - 1) / edge[i], n = (rows_b + edge[i] - 1) / edge[i];
        const int64_t tiles = batch * (symmetric ? m * (m + 1) / 2 : m * n);
        const double area = static_cast<double>(edge[i]) * edge[i];
        const double time = fmax(static_cast<double>((tiles + 255) / 256) * area / many[i], area / alone[i]);
        if (least == 0 || time < least) {
            least = time;
            best = edge[i];
        }
    }
    return best;
}

NewtonSpace carve_newton(int64_t rows, int64_t cols, int64_t batch, int32_t type, char *base) {
    NewtonSpace n{};
    n.planes = type == GNN_F32 ? 2 : 1;
    const int64_t s = rows < cols ? rows : cols, l = rows < cols ? cols : rows;
    n.s = (s + 63) / 64 * 64;
    n.l = (l + 63) / 64 * 64;
    n.plane_x = n.s * n.l;
    n.plane_a = n.s * n.s;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        off = (off + 255) & ~static_cast<size_t>(255);
        char *p = base ? base + off : nullptr;
        off += bytes;
        return p;
    };
    const size_t x = static_cast<size_t>(batch * n.planes * n.plane_x) * sizeof(f16);
    const size_t a = static_cast<size_t>(batch * n.planes * n.plane_a) * sizeof(f16);
    n.x = reinterpret_cast<f16 *>(take(x));
    n.xt[0] = reinterpret_cast<f16 *>(take(x));
    n.xt[1] = reinterpret_cast<f16 *>(take(x));
    n.a = reinterpret_cast<f16 *>(take(a));
    n.q = reinterpret_cast<f16 *>(take(a));
    n.partial = reinterpret_cast<double *>(take(static_cast<size_t>(batch) * kNormBlocks * 8));
    n.first = reinterpret_cast<float *>(take(static_cast<size_t>(batch) * 4));
    const size_t rest = n.planes == 1 ? static_cast<size_t>(batch * n.s) * 4 : 0;
    n.rest_a = reinterpret_cast<float *>(take(rest));
    n.rest_q = reinterpret_cast<float *>(take(rest));
    n.bytes = off;
    return n;
}

template <int TILE, int PL, typename TO>
hipError_t launch_tiles(ProductArgs p, int64_t batch, bool symmetric, hipStream_t s) {
    p.m_tiles = (p.rows_a + TILE - 1) / TILE;
    p.n_tiles = (p.rows_b + TILE - 1) / TILE;
    const int64_t tiles = symmetric ? static_cast<int64_t>(p.m_tiles) * (p.m_tiles + 1) / 2
                                    : static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    hipLaunchKernelGGL((k_newton_product<TILE, PL, TO>),
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(batch)), dim3(kThreads), 0,
                       s, p);
    return hipGetLastError();
}

template <int PL, typename TO>
hipError_t launch_product(const ProductArgs &p, int64_t batch, hipStream_t s) {
    const bool symmetric = p.what == kGram || p.what == kPoly;
    switch (tile_for(p.rows_a, p.rows_b, batch, symmetric, PL)) {
        case 192: return launch_tiles<PL == 1 ? 192 : 128, PL, TO>(p, batch, symmetric, s);
        case 128: return launch_tiles<128, PL, TO>(p, batch, symmetric, s);
        default: return launch_tiles<64, PL, TO>(p, batch, symmetric, s);
    }
}

template <int PL, typename T>
hipError_t run_newton(const NewtonArgs &a, hipStream_t s) {
    const NewtonSpace n = carve_newton(a.rows, a.cols, a.batch, a.type, a.ws);
    const bool wide = a.rows <= a.cols;
    const int64_t bx = PL * n.plane_x, ba = PL * n.plane_a;
    PrepArgs p{};
    p.g = a.g;
    p.rows = a.rows;
    p.cols = a.cols;
    p.ld = a.ld_g;
    p.batch_g = a.batch_g;
    p.partial = n.partial;
    const int64_t want = (a.rows + 3) / 4;
    p.blocks = static_cast<int32_t>(want < kNormBlocks ? want : kNormBlocks);
    p.eps = a.eps;
    p.first = n.first;
    p.same = wide ? n.x : n.xt[0];
    p.turned = wide ? n.xt[0] : n.x;
    p.ld_same = wide ? n.l : n.s;
    p.ld_turned = wide ? n.s : n.l;
    p.plane = n.plane_x;
    p.batch = bx;
    const unsigned nb = static_cast<unsigned>(a.batch);
    hipLaunchKernelGGL((k_norm_squares<T>), dim3(static_cast<unsigned>(p.blocks), nb),
                       dim3(kNormThreads), 0, s, p);
    const int64_t pr = wide ? n.s : n.l, pc = wide ? n.l : n.s;
    hipLaunchKernelGGL((k_first_planes<T, PL>),
                       dim3(static_cast<unsigned>(pc / 64), static_cast<unsigned>(pr / 64), nb),
                       dim3(kNormThreads), 0, s, p);
    hipError_t err = hipGetLastError();
    for (int step = 0; step < a.steps && err == hipSuccess; ++step) {
        const float *first = step == 0 ? n.first : nullptr;
        const bool last = step + 1 == a.steps;
        ProductArgs g{};
        g.what = kGram;
        g.a = g.b = n.x;
        g.ld_a = g.ld_b = g.k = n.l;
        g.plane_a = g.plane_b = n.plane_x;
        g.batch_a = g.batch_b = bx;
        g.c = g.t = n.a;
        g.ld_c = g.ld_t = n.s;
        g.plane_c = g.plane_t = n.plane_a;
        g.batch_c = g.batch_t = ba;
        g.rows_a = g.rows_b = static_cast<int32_t>(n.s);
        g.first = first;
        g.rest_a = n.rest_a;
        g.rest_q = n.rest_q;
        g.ld_rest = n.s;
        err = launch_product<PL, T>(g, a.batch, s);
        if (err != hipSuccess) return err;
        ProductArgs q = g;
        q.what = kPoly;
        q.a = q.b = n.a;
        q.ld_a = q.ld_b = q.k = n.s;
        q.plane_a = q.plane_b = n.plane_a;
        q.batch_a = q.batch_b = ba;
        q.c = q.t = n.q;
        q.ca = a.coefs[0];
        q.cb = a.coefs[1];
        q.cc = a.coefs[2];
        q.first = nullptr;
        err = launch_product<PL, T>(q, a.batch, s);
        if (err != hipSuccess) return err;
        ProductArgs y{};
        y.what = last ? kLast : kApply;
        y.a = n.xt[step & 1];
        y.ld_a = y.k = n.s;
        y.plane_a = n.plane_x;
        y.batch_a = bx;
        y.b = n.q;
        y.ld_b = n.s;
        y.plane_b = n.plane_a;
        y.batch_b = ba;
        y.c = n.xt[(step + 1) & 1];
        y.ld_c = n.s;
        y.plane_c = y.plane_t = n.plane_x;
        y.batch_c = y.batch_t = bx;
        y.t = n.x;
        y.ld_t = n.l;
        y.rows_a = static_cast<int32_t>(n.l);
        y.rows_b = static_cast<int32_t>(n.s);
        y.first = first;
        y.rest_a = n.rest_a;
        y.rest_q = n.rest_q;
        y.ld_rest = n.s;
        y.out = a.out;
        y.ld_out = a.ld_out;
        y.batch_out = a.batch_out;
        y.m = wide ? a.cols : a.rows;
        y.n = wide ? a.rows : a.cols;
        y.out_rows = wide ? 0 : 1;
        y.scale = a.scale;
        err = launch_product<PL, T>(y, a.batch, s);
    }
    return err;
}

}  // namespace

size_t newton_bytes(int64_t rows, int64_t cols, int64_t batch, int32_t type) {
    return carve_newton(rows, cols, batch, type, nullptr).bytes;
}

// The largest singular value that the steps can reach from [0, 1], and the largest of
// |a + b t + c t^2| on their squares; both bound the stored entries.
bool newton_in_range(const float *coefs, int steps) {
    const double a = coefs[0], b = coefs[1], c = coefs[2];
    if (!isfinite(a) || !isfinite(b) || !isfinite(c)) return false;
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        double next = 0.0, q = 0.0;
        auto look = [&](double s) {
            if (!(s >= 0 && s <= top)) return;
            const double t = s * s, v = a + b * t + c * t * t;
            next = fmax(next, fabs(s * v));
            q = fmax(q, fabs(v));
        };
        look(0.0);
        look(top);
        if (c != 0) {
            look(sqrt(fmax(0.0, -b / (2 * c))));                 // of a + b t + c t^2
            const double root = sqrt(fmax(0.0, 9 * b * b - 20 * a * c));
            look(sqrt(fmax(0.0, (-3 * b + root) / (10 * c))));   // of a s + b s^3 + c s^5
            look(sqrt(fmax(0.0, (-3 * b - root) / (10 * c))));
        } else if (b != 0) {
            look(sqrt(fmax(0.0, -a / (3 * b))));
        }
        if (!(next <= 3.0 && q <= 15.0)) return false;
        top = fmax(next, 1e-30);
    }
    return true;
}

hipError_t launch_newton(const NewtonArgs &a, hipStream_t s) {
    return a.type == GNN_F32 ? run_newton<2, float>(a, s) : run_newton<1, bf16>(a, s);
}

}  // namespace gnnmb
