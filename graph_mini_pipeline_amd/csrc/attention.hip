// Cross attention of packed query rows to the states of their own sequence, and its backward pass.
//
// Sequence b's queries are rows q_indptr[b] .. q_indptr[b+1], its states rows k_indptr[b] ..
// k_indptr[b+1] (the first k_count[b] of them).  With S = scale q k^T and, per query row,
// lse = log sum_j exp S_j, P_j = exp(S_j - lse):
//   out = P v;   D = dout . out,  dP = dout v^T,  dS = scale P (dP - D),
//   dq = dS k,  dk = dS^T q,  dv = P^T dout.
//
// The query heads that share states are taken together: a sequence's rows for one state head are its
// (query, head of the group) pairs, so a single token of a grouped model still fills a tile of rows,
// states are read once for the whole group, and dk and dv sum over the group by themselves.
//
// Tiles.  The 32 x 32 matrix instructions leave a lane one column and sixteen rows of the result, four
// at a time next to each other.  Products are turned so that the next one can take that as its
// operand as it is, without moving a value between lanes:
//   forward, dq:  S^T = k q^T (column = query row: running maximum and sum are per-lane numbers),
//                 then out^T += v^T P^T and dq^T += k^T dS^T, the summed index being the states;
//   dk, dv:       S = q k^T (column = state), then dv^T += dout^T P and dk^T += q^T dS, the summed
//                 index being the query rows.
// The transposed operands v^T, k^T, dout^T, q^T come from row-major LDS tiles: for bf16 by the LDS
// reads that transpose 4 x 16 blocks, for fp32 by single words (its matrix instructions take one
// word a lane and are slower than the reads).  The order in which the summed index is laid over
// the instruction's slots is the result's own, the same for both operands.
//
// fp32 runs on the fp32 matrix instructions; bf16 on the bf16 ones, with P and dS rounded to bf16
// (a half step of 2^-8, the size of the rounding of the results; short sums of the gradients: as two
// bf16, 2^-16), everything else in fp32.
//
// What bounds it.  For bf16 with many rows, LDS: an operand read is 1 KB for one matrix instruction of 32
// cycles, four of them at once are the 128 bytes a cycle that a compute unit's LDS delivers, and the
// exponentials and the tiles' way into LDS come on top.  4 sequences of up to 1024 queries of 16 heads
// over 4, up to 2600 states of 128: forward 109 us (490 TFLOP/s), dq 109 us (730), dk and dv 208 us (510
// by four products).  For single tokens, the reading of k and v: 16 sequences over up to 16384 states
// of 4 x 128, 346 MB in 94 us (3.7 TB/s; a large copy reaches 4.9).  For fp32, the matrix
// instructions, of which a 32 x 32 x 2 takes 64 cycles.
#include <math.h>
#include <type_traits>

#include "learn.hpp"

namespace gnnmb {

namespace {

typedef vec<float, 16> f32x16;
typedef vec<float, 4> f32x4;
constexpr int kThreads = 256;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
struct Kind;
template <>
struct Kind<bf16> {
    static constexpr int kPiece = 8;     // elements of 16 bytes
};
template <>
struct Kind<float> {
    static constexpr int kPiece = 4;
};
template <typename T>
using Piece = vec<T, Kind<T>::kPiece>;

// acc += A B^T over the 2 x kPiece summed elements that the two lane halves hold.
__device__ __forceinline__ void mma(f32x16 &acc, Piece<bf16> a, Piece<bf16> b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &acc, Piece<float> a, Piece<float> b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], acc, 0, 0, 0);
}

// A row-major LDS tile of DP columns, in 16-byte pieces.  A row is one piece longer than its columns, so
// that the 32 rows which a read touches at the same piece spread over the banks, and every other
// distance within a tile is a constant.  Row r lies at place(r): the rows 4 h + 0..3 of every sixteen
// are four places apart, so that the 4 x 16 blocks of a transposing read, two beside each other, fill
// the 64 banks exactly.
__device__ __forceinline__ int place(int r) {
    return (r & ~15) | ((r & 3) << 2) | ((r >> 3 & 1) << 1) | (r >> 2 & 1);
}
template <typename T, int DP>
struct Tile {
    static constexpr int NP = DP / Kind<T>::kPiece;      // pieces per row
    static constexpr int kStride = NP + 1;
    static constexpr int pieces(int rows) { return rows * kStride; }
    Piece<T> *p;
    // piece c of row r
    __device__ __forceinline__ Piece<T> *at(int r, int c) const { return p + place(r) * kStride + c; }
    // element d of row 4 h, 4 h of a tile's first sixteen rows
    __device__ __forceinline__ T *quad(int h, int d) const {
        return reinterpret_cast<T *>(p + h * kStride) + d;
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Operands come from LDS through a ring of RING registers sets, each read RING steps before the matrix
// instructions that use it (left alone, the compiler reads one, waits for it, multiplies, and reads
// the next).  use(s, v) may carry other work, which the matrix instructions hide.
constexpr int kOthersMove = 0x406;      // scalar, vector and transcendental arithmetic may cross
template <int RING, int STEPS, typename V, typename L>
__device__ __forceinline__ void prime(V (&v)[RING], L load) {
#pragma unroll
    for (int s = 0; s < RING && s < STEPS; ++s) v[s] = load(s);
    __builtin_amdgcn_sched_barrier(0);
}
template <int RING, int STEPS, typename V, typename L, typename U>
__device__ __forceinline__ void stream(V (&v)[RING], L load, U use) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        use(s, v[s % RING]);
        if (s + RING < STEPS) v[s % RING] = load(s + RING);
        __builtin_amdgcn_sched_barrier(kOthersMove);
    }
}

// The transposed operand of acc[db] += (columns 32 db .. of the tile's rows row0 .. row0+31)^T p, p
// being a 32 x 32 result whose rows are those 32: kSteps steps, each with a read of its own.
template <typename T, int DP>
struct Turned;

template <int DP>
struct Turned<bf16, DP> {
    static constexpr int DB = DP / 32, kSteps = 2 * DB, kRing = 4;
    struct V {
        s16x4 lo, hi;
    };
    static __device__ __forceinline__ V load(const Tile<bf16, DP> &tile, int row0, int s) {
        const int lane = lane_id();
        // the transposing read: 16 lanes name a 4 x 16 block, 4 elements each, and get a column each;
        // a row's successor is four places on, the row eight below it two
        constexpr int kRow = Tile<bf16, DP>::kStride * 8;
        const int d = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        bf16 *at = tile.quad(lane >> 5, d) + ((lane & 15) >> 2) * 4 * kRow + (row0 + 16 * (s / DB)) * kRow +
                   32 * (s % DB);
        return V{__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at),
                 __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + 2 * kRow))};
    }
    Piece<bf16> b, low; // p's half that the current steps multiply, and what bf16 leaves of it
    template <bool LOW>
    __device__ __forceinline__ void use(f32x16 (&acc)[DB], const V &v, int s, const f32x16 &p) {
        if (s % DB == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = static_cast<bf16>(p[8 * (s / DB) + e]);
#pragma unroll
            for (int e = 0; LOW && e < 8; ++e)
                low[e] = static_cast<bf16>(p[8 * (s / DB) + e] - static_cast<float>(b[e]));
        }
        const vec<short, 8> a = __builtin_shufflevector(v.lo, v.hi, 0, 1, 2, 3, 4, 5, 6, 7);
        mma(acc[s % DB], __builtin_bit_cast(Piece<bf16>, a), b);
        if (LOW) mma(acc[s % DB], __builtin_bit_cast(Piece<bf16>, a), low);
    }
};

template <int DP>
struct Turned<float, DP> {
    static constexpr int DB = DP / 32, kSteps = 16, kRing = 4;
    struct V {
        float a[DB];
    };
    static __device__ __forceinline__ V load(const Tile<float, DP> &tile, int row0, int s) {
        const int lane = lane_id();
        // row 8 (s / 4) + 4 half + s % 4
        const float *at = tile.quad(lane >> 5, lane & 31) +
                          (row0 + 16 * (s >> 3) + 2 * (s >> 2 & 1) + 4 * (s & 3)) * Tile<float, DP>::kStride * 4;
        V v;
#pragma unroll
        for (int db = 0; db < DB; ++db) v.a[db] = at[32 * db];
        return v;
    }
    template <bool LOW>
    __device__ __forceinline__ void use(f32x16 (&acc)[DB], const V &v, int s, const f32x16 &p) {
#pragma unroll
        for (int db = 0; db < DB; ++db)
            acc[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(v.a[db], p[s], acc[db], 0, 0, 0);
    }
};

struct Seq {
    int64_t q0, nq;      // first query row, queries
    int64_t k0, nk;      // first state row, states that count
    int64_t span;        // state rows, counted or not
};

__device__ __forceinline__ int64_t clamped(int64_t x, int64_t lo, int64_t hi) {
    return x < lo ? lo : (x < hi ? x : hi);
}

__device__ __forceinline__ Seq sequence(const AttendArgs &a, int64_t b) {
    Seq s;
    const int64_t q0 = a.q_indptr[b], q1 = a.q_indptr[b + 1];
    const int64_t k0 = a.k_indptr[b], k1 = a.k_indptr[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k)
        set_status(a.status, GNN_ERR_OUT_OF_RANGE);
    s.q0 = clamped(q0, 0, a.n_q);
    s.nq = clamped(q1, s.q0, a.n_q) - s.q0;
    s.k0 = clamped(k0, 0, a.n_k);
    s.span = clamped(k1, s.k0, a.n_k) - s.k0;
    if (s.nq > a.max_q || s.span > a.max_k) {
        set_status(a.status, GNN_ERR_CAPACITY);
        if (s.nq > a.max_q) s.nq = a.max_q;
        if (s.span > a.max_k) s.span = a.max_k;
    }
    s.nk = a.k_count ? clamped(a.k_count[b], 0, s.span) : s.span;
    return s;
}

// A row of a group: its position in a [n_q, heads, d] tensor of row stride ld.
struct GroupRow {
    int64_t pos;    // query row
    int32_t head;
};
__device__ __forceinline__ GroupRow group_row(const AttendArgs &a, const Seq &s, int hk, int64_t r) {
    GroupRow g;
    const uint32_t q = fast_div(static_cast<uint32_t>(r), a.by_group);
    g.pos = s.q0 + q;
    g.head = hk * a.group + static_cast<int32_t>(static_cast<uint32_t>(r) - q * a.group);
    return g;
}

// Loads R rows of DP columns into registers, and puts them into a tile a turn later, columns at or past d
// as zeros and rows at or past `rows` as zeros too or as row 0 (only there, so that nothing waits for
// the loads before).  at(r) is row r's distance in elements from `base`, which is the same for all
// threads, so that an address is a scalar pair and one 32-bit register (a tile's rows span fewer than
// 2^31 bytes); row 0 exists.  The first 256 threads of the workgroup call it.
template <typename T, int DP, int R>
struct Stage {
    static constexpr int NP = DP / Kind<T>::kPiece;
    static constexpr int kAll = R * NP;
    static constexpr int N = (kAll + kThreads - 1) / kThreads;     // the last turn may be a part of one
    Piece<T> v[N];
    template <typename F>
    __device__ __forceinline__ void load(const T *base, int64_t rows, int d, F at) {
        const char *from = reinterpret_cast<const char *>(base);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * kThreads + static_cast<int>(threadIdx.x);
            const int r = e / NP, c = e % NP * Kind<T>::kPiece;
            // every load is made, of a place that exists, so that none waits for a branch
            const uint32_t off = (at(r < rows ? r : 0) + (c < d ? c : 0)) * static_cast<uint32_t>(sizeof(T));
            v[i] = *reinterpret_cast<const typename loose<T, Kind<T>::kPiece>::type *>(from + off);
        }
    }
    __device__ __forceinline__ void put(const Tile<T, DP> &tile, int64_t rows, int d) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * kThreads + static_cast<int>(threadIdx.x);
            const int r = e / NP, c = e % NP;
            const Piece<T> x = r < rows && c * Kind<T>::kPiece < d ? v[i] : Piece<T>(static_cast<T>(0.f));
            if (kAll % kThreads == 0 || e < kAll) *tile.at(r, c) = x;
        }
    }
};

// One row as the operand that stays in registers: lane % 32 is the row, the two halves alternate pieces.
template <typename T, int DP>
struct RowPieces {
    static constexpr int KK = DP / Kind<T>::kPiece / 2;
    Piece<T> v[KK];
    __device__ __forceinline__ void load(const T *row, bool there, int d) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int c = (2 * kk + (lane_id() >> 5)) * Kind<T>::kPiece;
            const Piece<T> x =
                *reinterpret_cast<const typename loose<T, Kind<T>::kPiece>::type *>(row + (c < d ? c : 0));
            v[kk] = there && c < d ? x : Piece<T>(static_cast<T>(0.f));
        }
    }
};

// Step s of the product of tile rows row0 .. row0+31 with the registers' rows.
template <typename T>
constexpr int row_ring() {
    return sizeof(T) == 2 ? 4 : 3;      // an fp32 step is four long instructions
}
template <typename T, int DP>
__device__ __forceinline__ Piece<T> row_piece(const Tile<T, DP> &tile, int row0, int s) {
    const int lane = lane_id();
    return tile.at(lane & 31, lane >> 5)[row0 * Tile<T, DP>::kStride + 2 * s];
}

// Writes the four consecutive elements d0 .. d0+3 of a row (of d elements, a multiple of 8).
template <typename T>
__device__ __forceinline__ void put4(T *row, int d0, int d, f32x4 v) {
    if (d0 < d) store_f32<T, 4>(row + d0, v);
}

// A sequence's states (or rows) are split into as many parts of at most `per` as they need (an empty
// sequence has one part, which is empty), of equal length up to a multiple of `unit`.
__device__ __forceinline__ int64_t parts_of(int64_t n, int64_t per) {
    return n <= per ? 1 : (n + per - 1) / per;
}
__device__ __forceinline__ void part_range(int64_t n, int64_t per, int part, int unit, int64_t &begin,
                                           int64_t &end) {
    int64_t len = per;
    if (n > per) {
        const int64_t parts = (n + per - 1) / per;
        len = ((n + parts - 1) / parts + unit - 1) / unit * unit;
    }
    begin = len * part < n ? len * part : n;
    end = begin + len < n ? begin + len : n;
}

// States per wavefront and turn.
template <typename T, int WK>
constexpr int keys_per_wave() {
    return sizeof(T) == 2 && WK == 1 ? 64 : 32;
}

// Wavefronts that share the states where rows are few: four, or two where four wavefronts' tiles, twice,
// exceed the LDS.
template <typename T, int DP>
constexpr int sharing() {
    return sizeof(T) * DP <= 256 ? 4 : 2;
}

// ---- forward --------------------------------------------------------------------------------------
//
// WQ wavefronts take 32 rows each of a tile of rows, WK wavefronts share the states among them (for
// a sequence's few rows: four wavefronts read four times as many states a turn).  splits > 1: the
// states are shared among workgroups as well, whose sums the combining kernel joins.
template <typename T, int DP, int WQ, int WK>
__global__ __launch_bounds__(kThreads, WK == 1 ? 2 : 1) void k_attend(AttendArgs a) {
    constexpr int KW = keys_per_wave<T, WK>(), BK = KW * WK, BQ = 32 * WQ, KB = KW / 32;
    constexpr int DB = DP / 32;
    typedef Tile<T, DP> Tl;
    typedef Turned<T, DP> Tu;
    // two pairs of tiles of k and v: one is read while the next one is on its way
    constexpr int kPair = 2 * Tl::pieces(BK);
    __shared__ Piece<T> smem[2 * kPair];
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t rows = s.nq * a.group, r0 = (a.first_block + blockIdx.x) * BQ;
    if (r0 >= rows || split >= parts_of(s.nk, a.per)) return;      // whole workgroup
    int64_t kb, ke;
    part_range(s.nk, a.per, split, BK, kb, ke);
    const int lane = lane_id(), w = threadIdx.x >> 6, wq = w / WK, wk = w % WK;
    const int64_t r = r0 + wq * 32 + (lane & 31);
    const GroupRow me = group_row(a, s, hk, r < rows ? r : rows - 1);
    RowPieces<T, DP> q;
    q.load(static_cast<const T *>(a.q) + me.pos * a.ld_q + me.head * a.d, r < rows, a.d);

    const T *kp = static_cast<const T *>(a.k) + s.k0 * a.ld_k + hk * a.d;
    const T *vp = static_cast<const T *>(a.v) + s.k0 * a.ld_v + hk * a.d;
    f32x16 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) o[i] = f32x16(0.f);
    float top = -INFINITY, sum = 0.f;       // of scale * log2(e) * S
    const auto k_row = [&](int i) { return static_cast<uint32_t>(i) * static_cast<uint32_t>(a.ld_k); };
    const auto v_row = [&](int i) { return static_cast<uint32_t>(i) * static_cast<uint32_t>(a.ld_v); };
    Stage<T, DP, BK> sk, sv;
    const auto load = [&](int64_t at) __attribute__((always_inline)) {
        sk.load(kp + at * a.ld_k, ke - at, a.d, k_row);
        sv.load(vp + at * a.ld_v, ke - at, a.d, v_row);
    };
    const auto put = [&](Piece<T> *pair, int64_t at) __attribute__((always_inline)) {
        sk.put(Tl{pair}, ke - at, a.d);
        sv.put(Tl{pair + kPair / 2}, ke - at, a.d);
        __syncthreads();
    };
    const auto turn = [&](Piece<T> *pair, Piece<T> *next, int64_t k0) {
        const Tl tk{pair}, tv{pair + kPair / 2};
        const int64_t k1 = k0 + BK;
        if (k1 < ke) load(k1);
        constexpr int KK = RowPieces<T, DP>::KK, kR = row_ring<T>();
        f32x16 x[KB];
        float most = -INFINITY;
        const auto settle = [&](int b, int i) {       // the scaled score, -inf past the end
            x[b][i] *= a.scale2;
            if (k1 > ke && k0 + wk * KW + b * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= ke)
                x[b][i] = -INFINITY;
            most = fmaxf(most, x[b][i]);
        };
        Piece<T> ring[kR];
        const auto piece = [&](int st) { return row_piece<T, DP>(tk, wk * KW + st / KK * 32, st % KK); };
        prime<kR, KB * KK>(ring, piece);
#pragma unroll
        for (int b = 0; b < KB; ++b) x[b] = f32x16(0.f);
        stream<kR, KB * KK>(ring, piece, [&](int st, const Piece<T> &v) {
            mma(x[st / KK], v, q.v[st % KK]);
            if (st >= KK) {                           // the block before, meanwhile
#pragma unroll
                for (int i = st % KK * 16 / KK; i < (st % KK + 1) * 16 / KK; ++i) settle(st / KK - 1, i);
            }
        });
        typename Tu::V turned[Tu::kRing];
        const auto column = [&](int st) {
            return Tu::load(tv, wk * KW + st / Tu::kSteps * 32, st % Tu::kSteps);
        };
        prime<Tu::kRing, KB * Tu::kSteps>(turned, column);
#pragma unroll
        for (int i = 0; i < 16; ++i) settle(KB - 1, i);
        most = fmaxf(most, __shfl_xor(most, 32, 64));
        most = fmaxf(most, top);
        const float base = most == -INFINITY ? 0.f : most;
        if (__any(most > top)) {     // the sums so far are kept relative to the largest so far
            const float keep = __builtin_amdgcn_exp2f(top - base);
            sum *= keep;
#pragma unroll
            for (int i = 0; i < DB; ++i) o[i] *= keep;
            top = most;
        }
        const auto weigh = [&](int b, int i) {
            x[b][i] = __builtin_amdgcn_exp2f(x[b][i] - base);
            sum += x[b][i];
        };
#pragma unroll
        for (int i = 0; i < 16; ++i) weigh(0, i);
        Tu tu;
        stream<Tu::kRing, KB * Tu::kSteps>(turned, column, [&](int st, const typename Tu::V &v) {
            const int b = st / Tu::kSteps, t = st % Tu::kSteps;
            tu.template use<false>(o, v, t, x[b]);
            if (b + 1 < KB) {                         // the next block's weights, meanwhile
#pragma unroll
                for (int i = t * 16 / Tu::kSteps; i < (t + 1) * 16 / Tu::kSteps; ++i) weigh(b + 1, i);
            }
        });
        if (k1 < ke) put(next, k1);
    };
    if (kb < ke) {
        load(kb);
        put(smem, kb);
    }
    for (int64_t k0 = kb; k0 < ke; k0 += 2 * BK) {
        turn(smem, smem + kPair, k0);
        if (k0 + BK < ke) turn(smem + kPair, smem, k0 + BK);
    }
    sum += __shfl_xor(sum, 32, 64);
    if (WK > 1) {
        // join the wavefronts' sums: [WK - 1][32 rows][DP + 4] floats in the tiles' memory (DP sums, the
        // maximum and the weights' sum)
        constexpr int kRow = DP + 4;
        static_assert((WK - 1) * WQ * 32 * kRow * 4 <= static_cast<int>(sizeof(smem)), "join area");
        float *join = reinterpret_cast<float *>(smem) + (wq * (WK - 1) * 32 + (lane & 31)) * kRow;
        __syncthreads();
        if (wk > 0) {
            float *row = join + (wk - 1) * 32 * kRow;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<f32x4 *>(row + 32 * i + 8 * g + 4 * (lane >> 5)) =
                        f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
            if (lane < 32) {
                row[DP] = top;
                row[DP + 1] = sum;
            }
        }
        __syncthreads();
        if (wk > 0) return;
        for (int u = 0; u < WK - 1; ++u) {
            const float *row = join + u * 32 * kRow;
            const float t = row[DP], most = fmaxf(top, t);
            const float base = most == -INFINITY ? 0.f : most;
            const float mine = __builtin_amdgcn_exp2f(top - base), its = __builtin_amdgcn_exp2f(t - base);
            top = most;
            sum = sum * mine + row[DP + 1] * its;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 32 * i + 8 * g + 4 * (lane >> 5));
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][4 * g + e] = o[i][4 * g + e] * mine + v[e] * its;
                }
        }
    }
    if (r >= rows) return;
    const int64_t line = me.pos * a.heads + me.head;
    if (a.splits > 1) {
        float *part = a.part + (static_cast<int64_t>(split) * a.n_q * a.heads + line) * a.d;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                put4<float>(part, 32 * i + 8 * g + 4 * (lane >> 5), a.d,
                            f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]});
        if (lane < 32)
            a.part_stat[static_cast<int64_t>(split) * a.n_q * a.heads + line] = float2{top, sum};
        return;
    }
    const float each = sum == 0.f ? 0.f : 1.f / sum;
    T *out = static_cast<T *>(a.out) + me.pos * a.ld_out + me.head * a.d;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            put4<T>(out, 32 * i + 8 * g + 4 * (lane >> 5), a.d,
                    f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]} * each);
    if (a.lse && lane < 32) a.lse[line] = (top + log2f(sum)) * kLn2;
}

// Joins the splits of one row, a wavefront a row, two columns a lane.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attend_combine(AttendArgs a) {
    const Seq s = sequence(a, blockIdx.y);
    const int64_t line0 = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (line0 >= s.nq * a.heads) return;
    const int64_t line = s.q0 * a.heads + line0, all = a.n_q * a.heads;
    // each lane looks after one part's maximum and sum; kMaxSplits = 64
    const int parts = static_cast<int>(parts_of(s.nk, a.per));
    const int lane = lane_id();
    const float2 st = a.part_stat[(lane < parts ? lane : 0) * all + line];
    float top = lane < parts ? st.x : -INFINITY;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float base = top == -INFINITY ? 0.f : top;
    const float mine = lane < parts ? __builtin_amdgcn_exp2f(st.x - base) : 0.f;
    const float sum = wave_sum(lane < parts ? st.y * mine : 0.f);
    const int c = 2 * lane;
    float x = 0.f, y = 0.f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
        const float f = __shfl(mine, i, 64);
        const float2 v = *reinterpret_cast<const float2 *>(a.part + (i * all + line) * a.d + (c < a.d ? c : 0));
        x += v.x * f;
        y += v.y * f;
    }
    const int64_t pos = s.q0 + line0 / a.heads, head = line0 % a.heads;
    const float each = sum == 0.f ? 0.f : 1.f / sum;
    if (c < a.d) store_f32<T, 2>(static_cast<T *>(a.out) + pos * a.ld_out + head * a.d + c, vec<float, 2>{x * each, y * each});
    if (a.lse && lane == 0) a.lse[line] = (top + log2f(sum)) * kLn2;
}

// ---- backward -------------------------------------------------------------------------------------

// Where the statistics of a query row's head are kept: by state head, then as the group's rows.
__device__ __forceinline__ int64_t stat_at(const AttendArgs &a, int64_t pos, int32_t head) {
    const int32_t hk = static_cast<int32_t>(fast_div(static_cast<uint32_t>(head), a.by_group));
    return (hk * a.n_q + pos) * a.group + (head - hk * a.group);
}

// stat = {lse log2(e), D}; a row without weights (lse = -inf) gets +inf, which marks it.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attend_stat(AttendArgs a) {
    // eight lanes a row, 16 columns a lane
    const int64_t line = (a.first_block + blockIdx.x) * 32 + (threadIdx.x >> 3);
    if (line >= a.n_q * a.heads) return;
    const int64_t pos = line / a.heads, head = line - pos * a.heads;
    const T *o = static_cast<const T *>(a.out) + pos * a.ld_out + head * a.d;
    const T *g = static_cast<const T *>(a.dout) + pos * a.ld_dout + head * a.d;
    float sum = 0.f;
    for (int c = (threadIdx.x & 7) * 8; c < a.d; c += 64) {
        const vec<float, 8> x = load_f32<T, 8>(o + c) * load_f32<T, 8>(g + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[e];
    }
    sum += __shfl_xor(sum, 1, 64);
    sum += __shfl_xor(sum, 2, 64);
    sum += __shfl_xor(sum, 4, 64);
    if ((threadIdx.x & 7) == 0) {
        const float l = a.lse[line];
        a.stat[stat_at(a, pos, static_cast<int32_t>(head))] = float2{l == -INFINITY ? INFINITY : l * kLog2E, sum};
    }
}

// The bf16 that P and dS are rounded to leaves the gradients sqrt(2) times the error of their own
// rounding where the sums are long, and more where they are short (over 3 to 66 states 1.5 to 2 times):
// of a sequence with fewer than kLongSums rows or states, P and dS are multiplied as two bf16, which at
// 4 x 1024 queries of 16 heads over up to 2600 states took 579 us in place of 423.  The rule goes by the
// sequence's own lengths, so their precision does not depend on what else is in the call.
constexpr int64_t kLongSums = 512;
template <typename T>
__device__ __forceinline__ bool short_sums(const Seq &s, int64_t rows) {
    return sizeof(T) == 2 && (s.nk < kLongSums || rows < kLongSums);
}

// Over a single state the weight is 1 whatever q and k are: dS is zero.  P (dP - D) would leave the
// difference of two sums of the same products in other orders, rounding alone, so what dS is multiplied
// by last is zero there (a dS that is not finite still shows).
__device__ __forceinline__ float ds_factor(const AttendArgs &a, const Seq &s) {
    return s.nk == 1 ? 0.f : a.scale;
}

// Workgroups of k_attend_dq on a compute unit: two where their tiles and registers (256) allow.
template <typename T, int DP, int WK>
constexpr int dq_groups() {
    return (WK == 1 && sizeof(T) == 2) || sizeof(T) * DP * (WK == 1 ? 1 : 2) <= 256 ? 2 : 1;
}

// Dq of tiles of rows, as the forward kernel's.  Where a sequence's states fit one turn, D, which comes
// from the rounded out and another order of its sum, is put right by what the row of dS adds up to,
// which is zero; dk's kernel, which follows, reads it.
template <typename T, int DP, int WQ, int WK>
__global__ __launch_bounds__(kThreads, (dq_groups<T, DP, WK>())) void k_attend_dq(AttendArgs a) {
    constexpr int KW = 32, BK = KW * WK, BQ = 32 * WQ, DB = DP / 32;
    typedef Tile<T, DP> Tl;
    typedef Turned<T, DP> Tu;
    constexpr int kPair = 2 * Tl::pieces(BK);
    __shared__ Piece<T> smem[2 * kPair];
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t rows = s.nq * a.group, r0 = (a.first_block + blockIdx.x) * BQ;
    if (r0 >= rows || split >= parts_of(s.nk, a.per)) return;      // whole workgroup
    int64_t kb, ke;
    part_range(s.nk, a.per, split, BK, kb, ke);
    const int lane = lane_id(), w = threadIdx.x >> 6, wq = w / WK, wk = w % WK;
    const int64_t r = r0 + wq * 32 + (lane & 31);
    const GroupRow me = group_row(a, s, hk, r < rows ? r : rows - 1);
    const int64_t line = me.pos * a.heads + me.head;
    RowPieces<T, DP> q, g;
    q.load(static_cast<const T *>(a.q) + me.pos * a.ld_q + me.head * a.d, r < rows, a.d);
    g.load(static_cast<const T *>(a.dout) + me.pos * a.ld_dout + me.head * a.d, r < rows, a.d);
    const float2 st = a.stat[stat_at(a, me.pos, me.head)];
    const T *kp = static_cast<const T *>(a.k) + s.k0 * a.ld_k + hk * a.d;
    const T *vp = static_cast<const T *>(a.v) + s.k0 * a.ld_v + hk * a.d;
    f32x16 dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) dq[i] = f32x16(0.f);
    const auto k_row = [&](int i) { return static_cast<uint32_t>(i) * static_cast<uint32_t>(a.ld_k); };
    const auto v_row = [&](int i) { return static_cast<uint32_t>(i) * static_cast<uint32_t>(a.ld_v); };
    Stage<T, DP, BK> sk, sv;
    const auto load = [&](int64_t at) __attribute__((always_inline)) {
        sk.load(kp + at * a.ld_k, ke - at, a.d, k_row);
        sv.load(vp + at * a.ld_v, ke - at, a.d, v_row);
    };
    const auto put = [&](Piece<T> *pair, int64_t at) __attribute__((always_inline)) {
        sk.put(Tl{pair}, ke - at, a.d);
        sv.put(Tl{pair + kPair / 2}, ke - at, a.d);
        __syncthreads();
    };
    // (one_turn and low are constants: what the short sequences need would cost the others registers)
    const auto turn = [&](auto one_turn, auto low, Piece<T> *pair, Piece<T> *next, int64_t k0) __attribute__((always_inline)) {
        const Tl tk{pair}, tv{pair + kPair / 2};
        const int64_t k1 = k0 + BK;
        if (!one_turn.value && k1 < ke) load(k1);
        constexpr int KK = RowPieces<T, DP>::KK, kR = row_ring<T>();
        f32x16 x(0.f), dp(0.f);
        Piece<T> ring[kR];
        const auto piece = [&](int i) { return row_piece<T, DP>(i < KK ? tk : tv, wk * KW, i % KK); };
        prime<kR, 2 * KK>(ring, piece);
        typename Tu::V turned[Tu::kRing];
        const auto column = [&](int i) { return Tu::load(tk, wk * KW, i); };
        stream<kR, 2 * KK>(ring, piece, [&](int i, const Piece<T> &v) {
            if (i < KK) {
                mma(x, v, q.v[i]);
            } else {
                mma(dp, v, g.v[i - KK]);
#pragma unroll
                for (int j = (i - KK) * 16 / KK; j < (i - KK + 1) * 16 / KK; ++j)      // the weights, meanwhile
                    x[j] = __builtin_amdgcn_exp2f(x[j] * a.scale2 - st.x);      // (lse = +inf: 0)
            }
        });
        prime<Tu::kRing, Tu::kSteps>(turned, column);
        const auto past = [&](int i) {        // (in the last turn) a state past the end
            return k0 + wk * KW + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= ke;
        };
        dp -= st.y;
        if (one_turn.value) {
            float over = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) over += past(i) ? 0.f : x[i] * dp[i];
            over += __shfl_xor(over, 32, 64);
            dp -= over;       // (D + over, as one number, is rounded again)
            if (wk == 0 && lane < 32 && r < rows) a.stat[stat_at(a, me.pos, me.head)].y = st.y + over;
        }
        x *= dp;
        if (k1 > ke) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (past(i)) x[i] = 0.f;
        }
        Tu tu;
        stream<Tu::kRing, Tu::kSteps>(turned, column,
                                      [&](int i, const typename Tu::V &v) { tu.template use<low.value>(dq, v, i, x); });
        if (!one_turn.value && k1 < ke) put(next, k1);
    };
    if (kb < ke) {
        load(kb);
        put(smem, kb);
    }
    typedef std::bool_constant<sizeof(T) == 2> Low;
    const auto turns = [&](auto low) __attribute__((always_inline)) {
        for (int64_t k0 = kb; k0 < ke; k0 += 2 * BK) {
            turn(std::false_type{}, low, smem, smem + kPair, k0);
            if (k0 + BK < ke) turn(std::false_type{}, low, smem + kPair, smem, k0 + BK);
        }
    };
    if (kb < ke && s.nk <= KW)
        turn(std::true_type{}, Low{}, smem, smem + kPair, kb);
    else if (short_sums<T>(s, rows))
        turns(Low{});
    else
        turns(std::false_type{});
    if (WK > 1) {
        constexpr int kRow = DP + 4;
        static_assert((WK - 1) * WQ * 32 * kRow * 4 <= static_cast<int>(sizeof(smem)), "join area");
        float *join = reinterpret_cast<float *>(smem) + (wq * (WK - 1) * 32 + (lane & 31)) * kRow;
        __syncthreads();
        if (wk > 0) {
            float *row = join + (wk - 1) * 32 * kRow;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4 *>(row + 32 * i + 8 * j + 4 * (lane >> 5)) =
                        f32x4{dq[i][4 * j], dq[i][4 * j + 1], dq[i][4 * j + 2], dq[i][4 * j + 3]};
        }
        __syncthreads();
        if (wk > 0) return;
        for (int u = 0; u < WK - 1; ++u) {
            const float *row = join + u * 32 * kRow;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 32 * i + 8 * j + 4 * (lane >> 5));
#pragma unroll
                    for (int e = 0; e < 4; ++e) dq[i][4 * j + e] += v[e];
                }
        }
    }
    if (r >= rows) return;
    const float factor = ds_factor(a, s);
    T *out = static_cast<T *>(a.dq) + me.pos * a.ld_dq + me.head * a.d;
    float *part = a.part + (static_cast<int64_t>(split) * a.n_q * a.heads + line) * a.d;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 v = f32x4{dq[i][4 * j], dq[i][4 * j + 1], dq[i][4 * j + 2], dq[i][4 * j + 3]} * factor;
            const int d0 = 32 * i + 8 * j + 4 * (lane >> 5);
            if (a.splits > 1)
                put4<float>(part, d0, a.d, v);
            else
                put4<T>(out, d0, a.d, v);
        }
}

// dk and dv of 128 states, 32 a wavefront; splits > 1 shares the query rows among workgroups.  For bf16
// (SIDES = 2) four wavefronts take dv and four more dk of the same states: S is computed twice, 40
// products in place of 32, but each side's operands and sums leave room for two wavefronts per SIMD,
// whose waits overlap: the training step at 4 x 1024 queries of 16 heads over up to 2600 states takes
// 405 us (with one wavefront for both it took 466 where this took 421), this kernel 208 of it.  (At
// 227 us a turn took some 2700 cycles, 2200 of them LDS reads.)  For fp32, whose operands take twice the registers and whose
// products take sixteen times as long, one wavefront does both.
template <typename T, int DP, int SIDES>
__global__ __launch_bounds__(kThreads *SIDES, SIDES) void k_attend_dkv(AttendArgs a) {
    constexpr int BR = 32, DB = DP / 32;
    typedef Tile<T, DP> Tl;
    typedef Turned<T, DP> Tu;
    constexpr int kPair = 2 * Tl::pieces(BR);
    __shared__ Piece<T> smem[2 * kPair];
    __shared__ float sstat[2][2][BR];       // lse, then D
    __shared__ Piece<T> own[SIDES == 2 ? Tl::pieces(128) : 1];     // the states' v rows (dk's side)
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t c0 = (a.first_block + blockIdx.x) * 128;
    const int64_t rows = s.nq * a.group;
    if (c0 >= s.span || split >= parts_of(rows, a.per)) return;      // whole workgroup
    int64_t rb, re;
    part_range(rows, a.per, split, BR, rb, re);
    if (c0 >= s.nk) re = rb;                         // nothing counts
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool do_v = SIDES == 1 || w < 4, do_k = SIDES == 1 || w >= 4;
    const int64_t key = c0 + (w & 3) * 32 + (lane & 31);
    const bool counts = key < s.nk;
    const int64_t kr = s.k0 + (key < s.span ? key : 0);
    RowPieces<T, DP> k, v;
    k.load(static_cast<const T *>(a.k) + kr * a.ld_k + hk * a.d, counts, a.d);
    v.load(static_cast<const T *>(a.v) + kr * a.ld_v + hk * a.d, counts, a.d);
    const Tl tv{own};
    if (SIDES == 2 && do_k) {
        // read again in every turn (its registers are the sums'), by the wavefront that wrote them
#pragma unroll
        for (int i = 0; i < RowPieces<T, DP>::KK; ++i)
            *tv.at((w & 3) * 32 + (lane & 31), 2 * i + (lane >> 5)) = v.v[i];
        wave_lds_sync();
    }
    // the sums: dv and dk, or this side's
    f32x16 sums[2 / SIDES][DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        sums[0][i] = f32x16(0.f);
        sums[2 / SIDES - 1][i] = f32x16(0.f);
    }
    auto &dv = sums[0], &dk = sums[2 / SIDES - 1];
    // the statistics of this state head's rows lie next to each other
    const float2 *stat = a.stat + (static_cast<int64_t>(hk) * a.n_q + s.q0) * a.group;
    // dv's side, which has less to do, brings the tiles
    Stage<T, DP, BR> sq, sg;
    float2 st;
    const auto load = [&](int64_t r0) __attribute__((always_inline)) {
        if (!do_v) return;
        // the tile's first query row, and the rows' distances from its first head of the group
        const uint32_t p0 = fast_div(static_cast<uint32_t>(r0), a.by_group);
        const auto row = [&](int i, int64_t ld) {
            const uint32_t r = static_cast<uint32_t>(r0) + i, p = fast_div(r, a.by_group);
            return (p - p0) * static_cast<uint32_t>(ld) + (r - p * a.group) * static_cast<uint32_t>(a.d);
        };
        sq.load(static_cast<const T *>(a.q) + (s.q0 + p0) * a.ld_q + hk * a.group * a.d, re - r0, a.d,
                [&](int i) { return row(i, a.ld_q); });
        sg.load(static_cast<const T *>(a.dout) + (s.q0 + p0) * a.ld_dout + hk * a.group * a.d, re - r0,
                a.d, [&](int i) { return row(i, a.ld_dout); });
        const int64_t r = r0 + (threadIdx.x & (BR - 1));
        st = stat[r < re ? r : re - 1];
    };
    const auto put = [&](int pair, int64_t r0) __attribute__((always_inline)) {
        if (do_v) {
            // rows past the end are row 0's q again, without weights (zeros would make NaN of states
            // that are not finite), and zeros of dout (row 0's would make NaN of its infinities)
            sq.put(Tl{smem + pair * kPair}, BR, a.d);
            sg.put(Tl{smem + pair * kPair + kPair / 2}, re - r0, a.d);
            if (threadIdx.x < BR) {
                sstat[pair][0][threadIdx.x] = r0 + threadIdx.x < re ? st.x : INFINITY;
                sstat[pair][1][threadIdx.x] = st.y;
            }
        }
        __syncthreads();
    };
    const auto turn = [&](auto low, int pair, int64_t r0) __attribute__((always_inline)) {
        const Tl tq{smem + pair * kPair}, tg{smem + pair * kPair + kPair / 2};
        const int64_t r1 = r0 + BR;
        if (r1 < re) load(r1);
        constexpr int KK = RowPieces<T, DP>::KK, kR = row_ring<T>();
        f32x16 p(0.f), ds(0.f);
        Piece<T> ring[kR];
        const auto piece = [&](int i) { return row_piece<T, DP>(i < KK ? tq : tg, 0, i % KK); };
        // a step's row piece, and in dP's steps the piece of v
        struct Both {
            Piece<T> u, v;
        };
        const auto both = [&](int i) {
            Both x;
            x.u = piece(i);
            if (SIDES == 2 && i >= KK) x.v = row_piece<T, DP>(tv, (w & 3) * 32, i - KK);
            return x;
        };
        f32x4 lse[4], dd[4];      // rows 8 g + 4 half + 0..3
        const auto read_stat = [&](int which, f32x4 (&x)[4]) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                x[g] = *reinterpret_cast<const f32x4 *>(&sstat[pair][which][8 * g + 4 * (lane >> 5)]);
        };
        // lse = +inf, a row without weights: p = 0
        const auto weigh = [&](int j) {
            p[j] = __builtin_amdgcn_exp2f(p[j] * a.scale2 - lse[j >> 2][j & 3]);
        };
        const auto differ = [&](int j) { ds[j] = p[j] * (ds[j] - dd[j >> 2][j & 3]); };
        typename Tu::V turned[Tu::kRing];
        Tu tu;
        if (SIDES == 2 && do_v) {
            prime<kR, KK>(ring, piece);
            read_stat(0, lse);
            stream<kR, KK>(ring, piece, [&](int i, const Piece<T> &u) { mma(p, u, k.v[i]); });
            const auto column = [&](int i) { return Tu::load(tg, 0, i); };
            prime<Tu::kRing, Tu::kSteps>(turned, column);
#pragma unroll
            for (int j = 0; j < 16; ++j) weigh(j);
            stream<Tu::kRing, Tu::kSteps>(turned, column,
                                          [&](int i, const typename Tu::V &u) { tu.template use<low.value>(dv, u, i, p); });
        } else {
            Both pairs[kR];
            prime<kR, 2 * KK>(pairs, both);
            read_stat(0, lse);
            stream<kR, 2 * KK>(pairs, both, [&](int i, const Both &x) {
                if (i < KK) {
                    mma(p, x.u, k.v[i]);
                } else {
                    mma(ds, x.u, SIDES == 2 ? x.v : v.v[i - KK]);
#pragma unroll
                    for (int j = (i - KK) * 16 / KK; j < (i - KK + 1) * 16 / KK; ++j) weigh(j);   // meanwhile
                }
            });
            constexpr int kSteps = (3 - SIDES) * Tu::kSteps, kFirst = kSteps - Tu::kSteps;
            const auto column = [&](int i) {
                return Tu::load(i < kFirst ? tg : tq, 0, i % Tu::kSteps);
            };
            read_stat(1, dd);
            prime<Tu::kRing, kSteps>(turned, column);
            if (SIDES == 2) {
#pragma unroll
                for (int j = 0; j < 16; ++j) differ(j);
            }
            stream<Tu::kRing, kSteps>(turned, column, [&](int i, const typename Tu::V &u) {
                if (i < kFirst) {
                    tu.template use<low.value>(dv, u, i, p);
#pragma unroll
                    for (int j = i * 16 / Tu::kSteps; j < (i + 1) * 16 / Tu::kSteps; ++j) differ(j);
                } else {
                    tu.template use<low.value>(dk, u, i - kFirst, ds);
                }
            });
        }
        if (r1 < re) put(pair ^ 1, r1);
    };
    if (rb < re) {
        load(rb);
        put(0, rb);
    }
    const auto turns = [&](auto low) __attribute__((always_inline)) {
        for (int64_t r0 = rb; r0 < re; r0 += 2 * BR) {
            turn(low, 0, r0);
            if (r0 + BR < re) turn(low, 1, r0 + BR);
        }
    };
    if (short_sums<T>(s, rows))
        turns(std::bool_constant<sizeof(T) == 2>{});
    else
        turns(std::false_type{});
    if (key >= s.span) return;
    // a state past the count has no gradient
    const int64_t line = kr * a.kv + hk, all = a.n_k * a.kv;
    float *part = a.part + (static_cast<int64_t>(split) * all + line) * 2 * a.d;
    const auto write = [&](const f32x16 (&sum)[DB], float factor, T *to, float *part_to) {
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 x{sum[i][4 * j], sum[i][4 * j + 1], sum[i][4 * j + 2], sum[i][4 * j + 3]};
                x = counts ? x * factor : f32x4(0.f);
                const int d0 = 32 * i + 8 * j + 4 * (lane >> 5);
                if (a.splits > 1)
                    put4<float>(part_to, d0, a.d, x);
                else
                    put4<T>(to, d0, a.d, x);
            }
    };
    if (do_k) write(dk, ds_factor(a, s), static_cast<T *>(a.dk) + kr * a.ld_dk + hk * a.d, part);
    if (do_v) write(dv, 1.f, static_cast<T *>(a.dv) + kr * a.ld_dv + hk * a.d, part + a.d);
}

// What the reducing kernel takes: the splits of the states' sums, whose partial sums lie at part_kv, and
// those of dq (0: none to add).
struct ReduceArgs {
    int64_t dq_per, dkv_per;
    const float *part_kv;
    int32_t dq, dkv;
};

// Adds the splits of dq and (the grid's second layer, or the only one) of dk and dv.  A sequence's
// partial sums of one split are one stretch of memory: kReduceFours pieces of four a thread.
constexpr int kReduceFours = 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attend_reduce(AttendArgs a, ReduceArgs z) {
    const bool states = z.dkv && (!z.dq || blockIdx.z == 1);
    const Seq s = sequence(a, blockIdx.y);
    const int64_t first = states ? s.k0 : s.q0;
    const uint32_t per = states ? a.kv : a.heads;               // lines of a row
    const uint32_t fours = (states ? 2 * a.d : a.d) / 4;        // pieces of a line
    const int64_t count = (states ? s.span : s.nq) * per * fours;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kReduceFours) + threadIdx.x;
    if (static_cast<int64_t>(blockIdx.x) * (kThreads * kReduceFours) >= count) return;
    const int64_t all = (states ? a.n_k : a.n_q) * per * fours;
    const f32x4 *part = reinterpret_cast<const f32x4 *>(states ? z.part_kv : a.part) + first * per * fours;
    const int parts = states ? static_cast<int>(parts_of(s.nq * a.group, z.dkv_per))
                             : static_cast<int>(parts_of(s.nk, z.dq_per));
    f32x4 sum[kReduceFours];
#pragma unroll
    for (int u = 0; u < kReduceFours; ++u) sum[u] = f32x4(0.f);
#pragma unroll 2
    for (int i = 0; i < parts; ++i)
#pragma unroll
        for (int u = 0; u < kReduceFours; ++u) {
            const int64_t f = f0 + u * kThreads;
            sum[u] += part[i * all + (f < count ? f : 0)];
        }
#pragma unroll
    for (int u = 0; u < kReduceFours; ++u) {
        const int64_t f = f0 + u * kThreads;
        if (f >= count) continue;
        const int64_t line = f / fours;
        const int c = static_cast<int>(f - line * fours) * 4;
        const int64_t pos = line / per, head = line - pos * per, row = first + pos;
        T *to;
        if (!states)
            to = static_cast<T *>(a.dq) + row * a.ld_dq + head * a.d + c;
        else if (c < a.d)
            to = static_cast<T *>(a.dk) + row * a.ld_dk + head * a.d + c;
        else
            to = static_cast<T *>(a.dv) + row * a.ld_dv + head * a.d + c - a.d;
        store_f32<T, 4>(to, sum[u]);
    }
}

// ---- host -------------------------------------------------------------------------------------------

constexpr int64_t kWantGroups = 256;      // a workgroup per compute unit: more, for which states have to be
                                          // split further, cost more in partial sums than they even out
constexpr int64_t kFewTiles = 256;        // fewer tiles of 128 rows than compute units: tiles of 32
constexpr int64_t kMaxSplits = 64;        // one lane each in the combining kernel

// The plan of a call, from its host-side sizes alone.
struct Plan {
    bool few;                 // tiles of few rows, the wavefronts share the states
    int64_t q_tiles, k_tiles; // at least one: what is wrong with the indptrs or bounds is reported by the kernels
    int splits, dkv_splits;   // of the states (forward, dq) and of the rows (dk, dv)
    int64_t per, dkv_per;     // their lengths
    size_t stat, part_stat, part, part_kv, bytes;      // byte offsets
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Splits `length` among workgroups until `groups` of them times the splits fill the card, in parts of
// whole multiples of `least`.
void pick_splits(int64_t groups, int64_t length, int64_t least, int &splits, int64_t &per) {
    int64_t s = groups < 1 ? 1 : ceil_div(kWantGroups, groups);
    if (s > kMaxSplits) s = kMaxSplits;
    if (s < 1) s = 1;
    per = ceil_div(ceil_div(length, s), least) * least;
    if (per < least) per = least;
    splits = length <= per ? 1 : static_cast<int>(ceil_div(length, per));
}

Plan plan_for(const AttendArgs &a, bool backward) {
    Plan p{};
    const int64_t rows = a.max_q * a.group;
    const int64_t side = a.n_seq * a.kv;
    p.few = rows <= 32 || side * ceil_div(rows, 128) < kFewTiles;
    // (sharing(): two wavefronts' rows for wide fp32 heads)
    const int few_rows = a.type == GNN_F32 && a.d > 64 ? 64 : 32;
    p.q_tiles = ceil_div(rows, p.few ? few_rows : 128);
    p.k_tiles = ceil_div(a.max_k, 128);
    pick_splits(side * p.q_tiles, a.max_k, p.few ? 128 : 256, p.splits, p.per);
    pick_splits(side * p.k_tiles, rows, 128, p.dkv_splits, p.dkv_per);
    if (p.q_tiles < 1) p.q_tiles = 1;
    if (p.k_tiles < 1) p.k_tiles = 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    const size_t lines = static_cast<size_t>(a.n_q) * a.heads;
    if (backward) p.stat = take(lines * 8);
    const size_t part = p.splits > 1 ? lines * a.d * 4 * p.splits : 0;
    if (p.splits > 1) p.part_stat = take(lines * 8 * p.splits);
    p.part = take(part);
    if (backward && p.dkv_splits > 1)
        p.part_kv = take(static_cast<size_t>(a.n_k) * a.kv * 2 * a.d * 4 * p.dkv_splits);
    p.bytes = off < 256 ? 256 : off;
    return p;
}

#define TRY_LAUNCH(call)                       \
    do {                                       \
        const hipError_t err = (call);         \
        if (err != hipSuccess) return err;     \
    } while (0)

template <typename T, int DP>
hipError_t forward(AttendArgs a, const Plan &p, hipStream_t s) {
    a.splits = p.splits;
    a.per = p.per;
    const unsigned y = static_cast<unsigned>(a.kv * p.splits), z = static_cast<unsigned>(a.n_seq);
    TRY_LAUNCH(launch_pieces(p.q_tiles, kThreads, [&](int64_t first, unsigned x) {
        a.first_block = first;
        if (p.few)
            hipLaunchKernelGGL((k_attend<T, DP, 4 / sharing<T, DP>(), sharing<T, DP>()>), dim3(x, y, z),
                               dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((k_attend<T, DP, 4, 1>), dim3(x, y, z), dim3(kThreads), 0, s, a);
    }));
    // (a call with splits has few tiles, and so few rows)
    if (p.splits > 1)
        hipLaunchKernelGGL((k_attend_combine<T>),
                           dim3(static_cast<unsigned>(ceil_div(a.max_q * a.heads, 4)), z), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

// Each kernel reads what the one before left: none is enqueued after one that failed.
template <typename T, int DP>
hipError_t backward(AttendArgs a, const Plan &p, hipStream_t s) {
    const unsigned z = static_cast<unsigned>(a.n_seq);
    TRY_LAUNCH(launch_pieces(ceil_div(a.n_q * a.heads, 32), kThreads, [&](int64_t first, unsigned x) {
        a.first_block = first;
        hipLaunchKernelGGL((k_attend_stat<T>), dim3(x), dim3(kThreads), 0, s, a);
    }));
    a.splits = p.splits;
    a.per = p.per;
    TRY_LAUNCH(launch_pieces(p.q_tiles, kThreads, [&](int64_t first, unsigned x) {
        a.first_block = first;
        const dim3 grid(x, static_cast<unsigned>(a.kv * a.splits), z);
        if (p.few)
            hipLaunchKernelGGL((k_attend_dq<T, DP, 4 / sharing<T, DP>(), sharing<T, DP>()>), grid, dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((k_attend_dq<T, DP, 4, 1>), grid, dim3(kThreads), 0, s, a);
    }));
    float *const part_kv = reinterpret_cast<float *>(a.ws + p.part_kv);
    AttendArgs b = a;
    b.splits = p.dkv_splits;
    b.per = p.dkv_per;
    b.part = part_kv;
    constexpr int kSides = sizeof(T) == 2 ? 2 : 1;
    TRY_LAUNCH(launch_pieces(p.k_tiles, kThreads * kSides, [&](int64_t first, unsigned x) {
        b.first_block = first;
        hipLaunchKernelGGL((k_attend_dkv<T, DP, kSides>), dim3(x, static_cast<unsigned>(a.kv * b.splits), z),
                           dim3(kThreads * kSides), 0, s, b);
    }));
    ReduceArgs r{p.per, p.dkv_per, part_kv, a.max_q > 0 && p.splits > 1, a.max_k > 0 && p.dkv_splits > 1};
    if (r.dq || r.dkv) {
        const int64_t fq = r.dq ? a.max_q * a.heads * (a.d / 4) : 0;
        const int64_t fk = r.dkv ? a.max_k * a.kv * (a.d / 2) : 0;
        hipLaunchKernelGGL((k_attend_reduce<T>),
                           dim3(static_cast<unsigned>(ceil_div(fq > fk ? fq : fk, kThreads * kReduceFours)), z,
                                static_cast<unsigned>(r.dq + r.dkv)),
                           dim3(kThreads), 0, s, a, r);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t run(const AttendArgs &a, const Plan &p, bool back, hipStream_t s) {
    if (a.d <= 32) return back ? backward<T, 32>(a, p, s) : forward<T, 32>(a, p, s);
    if (a.d <= 64) return back ? backward<T, 64>(a, p, s) : forward<T, 64>(a, p, s);
    if (a.d <= 96) return back ? backward<T, 96>(a, p, s) : forward<T, 96>(a, p, s);
    return back ? backward<T, 128>(a, p, s) : forward<T, 128>(a, p, s);
}

}  // namespace

size_t attend_bytes(const AttendArgs &a, bool backward) { return plan_for(a, backward).bytes; }

hipError_t launch_attend(AttendArgs a, bool backward, char *ws, hipStream_t s) {
    if (a.n_seq == 0) return hipSuccess;
    const Plan p = plan_for(a, backward);
    a.by_group = make_fastdiv(static_cast<uint32_t>(a.group));
    a.scale2 = a.scale * kLog2E;
    a.ws = ws;
    a.stat = reinterpret_cast<float2 *>(ws + p.stat);
    a.part_stat = reinterpret_cast<float2 *>(ws + p.part_stat);
    a.part = reinterpret_cast<float *>(ws + p.part);
    return a.type == GNN_F32 ? run<float>(a, p, backward, s) : run<bf16>(a, p, backward, s);
}

}  // namespace gnnmb
