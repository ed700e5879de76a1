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
// (2^-9, the size of the rounding of the results), everything else in fp32.
#include <math.h>

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

// A row-major LDS tile of DP columns: 16-byte pieces, those of a row permuted by the row so that
// lanes reading the same piece of different rows use different banks.
template <typename T, int DP>
struct Tile {
    static constexpr int NP = DP / Kind<T>::kPiece;      // pieces per row
    static constexpr int kMask = (NP < 16 ? NP : 16) - 1;
    Piece<T> *p;
    __device__ __forceinline__ Piece<T> *at(int r, int c) const {
        return p + r * NP + (c ^ (r & kMask));
    }
    // element d of row r
    __device__ __forceinline__ T *element(int r, int d) const {
        return reinterpret_cast<T *>(at(r, d / Kind<T>::kPiece)) + d % Kind<T>::kPiece;
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// acc[db] += (columns 32 db .. of the tile's rows row0 .. row0+31)^T p, p being a 32 x 32 result
// whose rows are those 32.
template <int DP>
__device__ __forceinline__ void mma_turned(f32x16 (&acc)[DP / 32], const Tile<bf16, DP> &tile,
                                           int row0, const f32x16 &p) {
    const int lane = lane_id();
    // the transposing read: 16 lanes name a 4 x 16 block, 4 elements each, and get a column each
    const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int d = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Piece<bf16> b;
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = static_cast<bf16>(p[8 * t + e]);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)tile.element(row0 + 16 * t + r, 32 * db + d));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)tile.element(row0 + 16 * t + 8 + r, 32 * db + d));
            const vec<short, 8> a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            mma(acc[db], __builtin_bit_cast(Piece<bf16>, a), b);
        }
    }
}
template <int DP>
__device__ __forceinline__ void mma_turned(f32x16 (&acc)[DP / 32], const Tile<float, DP> &tile,
                                           int row0, const f32x16 &p) {
    const int lane = lane_id();
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int db = 0; db < DP / 32; ++db) {
                const float a = *tile.element(row0 + 8 * g + 4 * (lane >> 5) + e, 32 * db + (lane & 31));
                acc[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[4 * g + e], acc[db], 0, 0, 0);
            }
}

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

// Loads R rows of DP columns into registers, rows at or past `rows` and columns at or past d as zeros;
// put() stores them to the tile.  ptr(r) is row r's first element; row 0 exists.
template <typename T, int DP, int R>
struct Stage {
    static constexpr int NP = DP / Kind<T>::kPiece;
    static constexpr int N = R * NP / kThreads;
    Piece<T> v[N];
    template <typename F>
    __device__ __forceinline__ void load(int64_t rows, int d, F ptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * kThreads + static_cast<int>(threadIdx.x);
            const int r = e / NP, c = e % NP * Kind<T>::kPiece;
            // every load is made, of a place that exists, so that none waits for a branch
            const T *p = ptr(r < rows ? r : 0) + (c < d ? c : 0);
            const Piece<T> x = *reinterpret_cast<const typename loose<T, Kind<T>::kPiece>::type *>(p);
            v[i] = r < rows && c < d ? x : Piece<T>(static_cast<T>(0.f));
        }
    }
    __device__ __forceinline__ void put(const Tile<T, DP> &tile) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * kThreads + static_cast<int>(threadIdx.x);
            *tile.at(e / NP, e % NP) = v[i];
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

// The 32 x 32 product of tile rows row0 .. row0+31 with the registers' rows.
template <typename T, int DP>
__device__ __forceinline__ f32x16 product(const Tile<T, DP> &tile, int row0,
                                          const RowPieces<T, DP> &b) {
    f32x16 acc(0.f);
    const int lane = lane_id();
#pragma unroll
    for (int kk = 0; kk < RowPieces<T, DP>::KK; ++kk)
        mma(acc, *tile.at(row0 + (lane & 31), 2 * kk + (lane >> 5)), b.v[kk]);
    return acc;
}

// Writes the four consecutive elements d0 .. d0+3 of a row (of d elements, a multiple of 8).
template <typename T>
__device__ __forceinline__ void put4(T *row, int d0, int d, f32x4 v) {
    if (d0 < d) store_f32<T, 4>(row + d0, v);
}

// The states of one split of a sequence: [begin, end).
__device__ __forceinline__ void split_range(int64_t n, int split, int splits, int unit, int64_t &begin,
                                            int64_t &end) {
    int64_t per = (n + splits - 1) / splits;
    per = (per + unit - 1) / unit * unit;
    begin = per * split < n ? per * split : n;
    end = begin + per < n ? begin + per : n;
}

// States per wavefront and turn.
template <typename T, int WK>
constexpr int keys_per_wave() {
    return sizeof(T) == 2 && WK == 1 ? 64 : 32;
}

// ---- forward --------------------------------------------------------------------------------------
//
// WQ wavefronts take 32 rows each of a tile of rows, WK wavefronts share the states among them (for
// a sequence's few rows: four wavefronts read four times as many states a turn).  splits > 1: the
// states are shared among workgroups as well, whose sums the combining kernel joins.
template <typename T, int DP, int WQ, int WK>
__global__ __launch_bounds__(kThreads, 2) void k_attend(AttendArgs a) {
    constexpr int KW = keys_per_wave<T, WK>(), BK = KW * WK, BQ = 32 * WQ, KB = KW / 32;
    constexpr int DB = DP / 32;
    typedef Tile<T, DP> Tl;
    __shared__ Piece<T> smem[2 * BK * Tl::NP];
    const Tl tk{smem}, tv{smem + BK * Tl::NP};
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t rows = s.nq * a.group, r0 = static_cast<int64_t>(blockIdx.x) * BQ;
    if (r0 >= rows) return;      // whole workgroup
    const int lane = lane_id(), w = threadIdx.x >> 6, wq = w / WK, wk = w % WK;
    const int64_t r = r0 + wq * 32 + (lane & 31);
    const GroupRow me = group_row(a, s, hk, r < rows ? r : rows - 1);
    RowPieces<T, DP> q;
    q.load(static_cast<const T *>(a.q) + me.pos * a.ld_q + me.head * a.d, r < rows, a.d);

    int64_t kb, ke;
    split_range(s.nk, split, a.splits, BK, kb, ke);
    const T *kp = static_cast<const T *>(a.k) + s.k0 * a.ld_k + hk * a.d;
    const T *vp = static_cast<const T *>(a.v) + s.k0 * a.ld_v + hk * a.d;
    f32x16 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) o[i] = f32x16(0.f);
    float top = -INFINITY, sum = 0.f;       // of scale * log2(e) * S
    Stage<T, DP, BK> sk, sv;
    if (kb < ke) {
        sk.load(ke - kb, a.d, [&](int i) { return kp + (kb + i) * a.ld_k; });
        sv.load(ke - kb, a.d, [&](int i) { return vp + (kb + i) * a.ld_v; });
    }
    for (int64_t k0 = kb; k0 < ke; k0 += BK) {
        __syncthreads();          // the last turn's reads are done
        sk.put(tk);
        sv.put(tv);
        __syncthreads();
        const int64_t k1 = k0 + BK;
        if (k1 < ke) {
            sk.load(ke - k1, a.d, [&](int i) { return kp + (k1 + i) * a.ld_k; });
            sv.load(ke - k1, a.d, [&](int i) { return vp + (k1 + i) * a.ld_v; });
        }
        f32x16 x[KB];
        float most = -INFINITY;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            x[b] = product<T, DP>(tk, wk * KW + b * 32, q) * a.scale2;
            if (k1 > ke) {        // the last turn: states past the end
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + wk * KW + b * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= ke)
                        x[b][i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, x[b][i]);
        }
        most = fmaxf(most, __shfl_xor(most, 32, 64));
        most = fmaxf(most, top);
        const float base = most == -INFINITY ? 0.f : most;
        const float keep = __builtin_amdgcn_exp2f(top - base);
        top = most;
        sum *= keep;
#pragma unroll
        for (int i = 0; i < DB; ++i) o[i] *= keep;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[b][i] = __builtin_amdgcn_exp2f(x[b][i] - base);
                sum += x[b][i];
            }
            mma_turned<DP>(o, tv, wk * KW + b * 32, x[b]);
        }
    }
    sum += __shfl_xor(sum, 32, 64);
    if (WK > 1) {
        // join the wavefronts' sums: [WK - 1][32 rows][DP + 2] floats in the tiles' memory
        constexpr int kRow = DP + 4;
        static_assert((WK - 1) * 32 * kRow * 4 <= static_cast<int>(sizeof(smem)), "join area");
        float *join = reinterpret_cast<float *>(smem);
        __syncthreads();
        if (wk > 0) {
            float *row = join + ((wk - 1) * 32 + (lane & 31)) * kRow;
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
            const float *row = join + (u * 32 + (lane & 31)) * kRow;
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
    float top = -INFINITY;
    for (int i = 0; i < a.splits; ++i) top = fmaxf(top, a.part_stat[i * all + line].x);
    const float base = top == -INFINITY ? 0.f : top;
    const int c = 2 * lane_id();
    float sum = 0.f, x = 0.f, y = 0.f;
    for (int i = 0; i < a.splits; ++i) {
        const float2 st = a.part_stat[i * all + line];
        const float f = __builtin_amdgcn_exp2f(st.x - base);
        sum += st.y * f;
        if (c < a.d) {
            const float2 v = *reinterpret_cast<const float2 *>(a.part + (i * all + line) * a.d + c);
            x += v.x * f;
            y += v.y * f;
        }
    }
    const int64_t pos = s.q0 + line0 / a.heads, head = line0 % a.heads;
    const float each = sum == 0.f ? 0.f : 1.f / sum;
    if (c < a.d) store_f32<T, 2>(static_cast<T *>(a.out) + pos * a.ld_out + head * a.d + c, vec<float, 2>{x * each, y * each});
    if (a.lse && lane_id() == 0) a.lse[line] = (top + log2f(sum)) * kLn2;
}

// ---- backward -------------------------------------------------------------------------------------

// stat[line] = {lse log2(e), D}; a row without weights (lse = -inf) gets +inf, which marks it.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attend_stat(AttendArgs a) {
    // eight lanes a row, 16 columns a lane
    const int64_t line = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 3);
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
        a.stat[line] = float2{l == -INFINITY ? INFINITY : l * kLog2E, sum};
    }
}

template <typename T, int DP, int WQ, int WK>
__global__ __launch_bounds__(kThreads) void k_attend_dq(AttendArgs a) {
    constexpr int KW = 32, BK = KW * WK, BQ = 32 * WQ, DB = DP / 32;
    typedef Tile<T, DP> Tl;
    __shared__ Piece<T> smem[2 * BK * Tl::NP];
    const Tl tk{smem}, tv{smem + BK * Tl::NP};
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t rows = s.nq * a.group, r0 = static_cast<int64_t>(blockIdx.x) * BQ;
    if (r0 >= rows) return;      // whole workgroup
    const int lane = lane_id(), w = threadIdx.x >> 6, wq = w / WK, wk = w % WK;
    const int64_t r = r0 + wq * 32 + (lane & 31);
    const GroupRow me = group_row(a, s, hk, r < rows ? r : rows - 1);
    const int64_t line = me.pos * a.heads + me.head;
    RowPieces<T, DP> q, g;
    q.load(static_cast<const T *>(a.q) + me.pos * a.ld_q + me.head * a.d, r < rows, a.d);
    g.load(static_cast<const T *>(a.dout) + me.pos * a.ld_dout + me.head * a.d, r < rows, a.d);
    const float2 st = a.stat[line];
    int64_t kb, ke;
    split_range(s.nk, split, a.splits, BK, kb, ke);
    const T *kp = static_cast<const T *>(a.k) + s.k0 * a.ld_k + hk * a.d;
    const T *vp = static_cast<const T *>(a.v) + s.k0 * a.ld_v + hk * a.d;
    f32x16 dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) dq[i] = f32x16(0.f);
    Stage<T, DP, BK> sk, sv;
    if (kb < ke) {
        sk.load(ke - kb, a.d, [&](int i) { return kp + (kb + i) * a.ld_k; });
        sv.load(ke - kb, a.d, [&](int i) { return vp + (kb + i) * a.ld_v; });
    }
    for (int64_t k0 = kb; k0 < ke; k0 += BK) {
        __syncthreads();
        sk.put(tk);
        sv.put(tv);
        __syncthreads();
        const int64_t k1 = k0 + BK;
        if (k1 < ke) {
            sk.load(ke - k1, a.d, [&](int i) { return kp + (k1 + i) * a.ld_k; });
            sv.load(ke - k1, a.d, [&](int i) { return vp + (k1 + i) * a.ld_v; });
        }
        f32x16 x = product<T, DP>(tk, wk * KW, q);
        const f32x16 dp = product<T, DP>(tv, wk * KW, g);
        // states past the end: k and v are zeros there, and add nothing to dq
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = st.x == INFINITY ? 0.f
                                    : __builtin_amdgcn_exp2f(x[i] * a.scale2 - st.x) * (dp[i] - st.y);
        mma_turned<DP>(dq, tk, wk * KW, x);
    }
    if (WK > 1) {
        constexpr int kRow = DP + 4;
        static_assert((WK - 1) * 32 * kRow * 4 <= static_cast<int>(sizeof(smem)), "join area");
        float *join = reinterpret_cast<float *>(smem);
        __syncthreads();
        if (wk > 0) {
            float *row = join + ((wk - 1) * 32 + (lane & 31)) * kRow;
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
            const float *row = join + (u * 32 + (lane & 31)) * kRow;
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
    T *out = static_cast<T *>(a.dq) + me.pos * a.ld_dq + me.head * a.d;
    float *part = a.part + (static_cast<int64_t>(split) * a.n_q * a.heads + line) * a.d;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 v = f32x4{dq[i][4 * j], dq[i][4 * j + 1], dq[i][4 * j + 2], dq[i][4 * j + 3]} * a.scale;
            const int d0 = 32 * i + 8 * j + 4 * (lane >> 5);
            if (a.splits > 1)
                put4<float>(part, d0, a.d, v);
            else
                put4<T>(out, d0, a.d, v);
        }
}

// dk and dv of 128 states, 32 a wavefront; splits > 1 shares the query rows among workgroups.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void k_attend_dkv(AttendArgs a) {
    constexpr int BR = 32, DB = DP / 32;
    typedef Tile<T, DP> Tl;
    __shared__ Piece<T> smem[2 * BR * Tl::NP];
    __shared__ float2 sstat[BR];
    const Tl tq{smem}, tg{smem + BR * Tl::NP};
    const Seq s = sequence(a, blockIdx.z);
    const int hk = static_cast<int>(blockIdx.y) / a.splits, split = static_cast<int>(blockIdx.y) % a.splits;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 128;
    if (c0 >= s.span) return;      // whole workgroup
    const int lane = lane_id(), w = threadIdx.x >> 6;
    const int64_t key = c0 + w * 32 + (lane & 31);
    const bool counts = key < s.nk;
    const int64_t kr = s.k0 + (key < s.span ? key : 0);
    RowPieces<T, DP> k, v;
    k.load(static_cast<const T *>(a.k) + kr * a.ld_k + hk * a.d, counts, a.d);
    v.load(static_cast<const T *>(a.v) + kr * a.ld_v + hk * a.d, counts, a.d);
    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) dk[i] = dv[i] = f32x16(0.f);
    int64_t rb = 0, re = 0;
    if (c0 < s.nk) split_range(s.nq * a.group, split, a.splits, BR, rb, re);   // else: nothing counts
    Stage<T, DP, BR> sq, sg;
    float2 st{INFINITY, 0.f};
    auto load = [&](int64_t r0) {
        const auto q_row = [&](int i) {
            const GroupRow g = group_row(a, s, hk, r0 + i);
            return static_cast<const T *>(a.q) + g.pos * a.ld_q + g.head * a.d;
        };
        const auto g_row = [&](int i) {
            const GroupRow g = group_row(a, s, hk, r0 + i);
            return static_cast<const T *>(a.dout) + g.pos * a.ld_dout + g.head * a.d;
        };
        sq.load(re - r0, a.d, q_row);
        sg.load(re - r0, a.d, g_row);
        st = float2{INFINITY, 0.f};          // rows past the end: P = 0
        if (threadIdx.x < BR && r0 + threadIdx.x < re) {
            const GroupRow g = group_row(a, s, hk, r0 + threadIdx.x);
            st = a.stat[g.pos * a.heads + g.head];
        }
    };
    if (rb < re) load(rb);
    for (int64_t r0 = rb; r0 < re; r0 += BR) {
        __syncthreads();
        sq.put(tq);
        sg.put(tg);
        if (threadIdx.x < BR) sstat[threadIdx.x] = st;
        __syncthreads();
        if (r0 + BR < re) load(r0 + BR);
        f32x16 p = product<T, DP>(tq, 0, k);
        f32x16 ds = product<T, DP>(tg, 0, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 x = sstat[8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)];
            // a row without weights, or past the end: zero, also against states that are not finite
            const bool live = x.x != INFINITY;
            p[i] = live ? __builtin_amdgcn_exp2f(p[i] * a.scale2 - x.x) : 0.f;
            ds[i] = live ? p[i] * (ds[i] - x.y) : 0.f;
        }
        mma_turned<DP>(dv, tg, 0, p);
        mma_turned<DP>(dk, tq, 0, ds);
    }
    if (key >= s.span) return;
    // a state past the count has no gradient
    const int64_t line = kr * a.kv + hk, all = a.n_k * a.kv;
    float *part = a.part + (static_cast<int64_t>(split) * all + line) * 2 * a.d;
    T *ok = static_cast<T *>(a.dk) + kr * a.ld_dk + hk * a.d;
    T *ov = static_cast<T *>(a.dv) + kr * a.ld_dv + hk * a.d;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 x{dk[i][4 * j], dk[i][4 * j + 1], dk[i][4 * j + 2], dk[i][4 * j + 3]};
            f32x4 y{dv[i][4 * j], dv[i][4 * j + 1], dv[i][4 * j + 2], dv[i][4 * j + 3]};
            x = counts ? x * a.scale : f32x4(0.f);
            y = counts ? y : f32x4(0.f);
            const int d0 = 32 * i + 8 * j + 4 * (lane >> 5);
            if (a.splits > 1) {
                put4<float>(part, d0, a.d, x);
                put4<float>(part + a.d, d0, a.d, y);
            } else {
                put4<T>(ok, d0, a.d, x);
                put4<T>(ov, d0, a.d, y);
            }
        }
}

// Adds the splits of dq (states = 0) or of dk and dv (states = 1), a wavefront a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attend_reduce(AttendArgs a, int states) {
    const Seq s = sequence(a, blockIdx.y);
    const int64_t per = states ? a.kv : a.heads;
    const int64_t line0 = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (line0 >= (states ? s.span : s.nq) * per) return;
    const int64_t first = states ? s.k0 : s.q0;
    const int64_t line = first * per + line0;
    const int64_t all = (states ? a.n_k : a.n_q) * per;
    const int64_t pos = first + line0 / per, head = line0 % per;
    const int wide = states ? 2 * a.d : a.d;
    for (int c = 2 * lane_id(); c < wide; c += 128) {
        float x = 0.f, y = 0.f;
        for (int i = 0; i < a.splits; ++i) {
            const float2 v = *reinterpret_cast<const float2 *>(a.part + (i * all + line) * wide + c);
            x += v.x;
            y += v.y;
        }
        T *to;
        if (!states)
            to = static_cast<T *>(a.dq) + pos * a.ld_dq + head * a.d + c;
        else if (c < a.d)
            to = static_cast<T *>(a.dk) + pos * a.ld_dk + head * a.d + c;
        else
            to = static_cast<T *>(a.dv) + pos * a.ld_dv + head * a.d + c - a.d;
        store_f32<T, 2>(to, vec<float, 2>{x, y});
    }
}

// ---- host -------------------------------------------------------------------------------------------

constexpr int64_t kWantGroups = 1024;     // workgroups that fill the card
constexpr int64_t kMaxSplits = 64;

// The plan of a call, from its host-side sizes alone.
struct Plan {
    bool few;                 // at most 32 rows a sequence: the wavefronts share the states
    int64_t q_tiles, k_tiles;
    int splits, dq_splits, dkv_splits;
    size_t stat, part_stat, part, bytes;      // byte offsets
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int pick_splits(int64_t groups, int64_t length, int64_t least) {
    if (groups >= kWantGroups || groups < 1) return 1;
    int64_t s = ceil_div(kWantGroups, groups), most = length / least;
    if (s > most) s = most;
    if (s > kMaxSplits) s = kMaxSplits;
    return static_cast<int>(s < 1 ? 1 : s);
}

Plan plan_for(const AttendArgs &a, bool backward) {
    Plan p{};
    const int64_t rows = a.max_q * a.group;
    p.few = rows <= 32;
    p.q_tiles = ceil_div(rows, p.few ? 32 : 128);
    p.k_tiles = ceil_div(a.max_k, 128);
    const int64_t side = a.n_seq * a.kv;
    p.splits = p.dq_splits = pick_splits(side * p.q_tiles, a.max_k, 256);
    p.dkv_splits = pick_splits(side * p.k_tiles, rows, 128);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    const size_t lines = static_cast<size_t>(a.n_q) * a.heads;
    if (backward) p.stat = take(lines * 8);
    size_t part = p.splits > 1 ? lines * a.d * 4 * p.splits : 0;
    if (p.splits > 1) p.part_stat = take(lines * 8 * p.splits);
    if (backward && p.dkv_splits > 1) {
        const size_t kv = static_cast<size_t>(a.n_k) * a.kv * 2 * a.d * 4 * p.dkv_splits;
        part = kv > part ? kv : part;
    }
    p.part = take(part);
    p.bytes = off < 256 ? 256 : off;
    return p;
}

template <typename T, int DP>
hipError_t forward(AttendArgs a, const Plan &p, hipStream_t s) {
    a.splits = p.splits;
    const dim3 grid(static_cast<unsigned>(p.q_tiles), static_cast<unsigned>(a.kv * p.splits),
                    static_cast<unsigned>(a.n_seq));
    if (p.few)
        hipLaunchKernelGGL((k_attend<T, DP, 1, 4>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_attend<T, DP, 4, 1>), grid, dim3(kThreads), 0, s, a);
    if (p.splits > 1)
        hipLaunchKernelGGL((k_attend_combine<T>),
                           dim3(static_cast<unsigned>(ceil_div(a.max_q * a.heads, 4)),
                                static_cast<unsigned>(a.n_seq)),
                           dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <typename T, int DP>
hipError_t backward(AttendArgs a, const Plan &p, hipStream_t s) {
    const unsigned z = static_cast<unsigned>(a.n_seq);
    if (a.n_q > 0)
        hipLaunchKernelGGL((k_attend_stat<T>),
                           dim3(static_cast<unsigned>(ceil_div(a.n_q * a.heads, 32))),
                           dim3(kThreads), 0, s, a);
    if (a.max_q > 0) {
        a.splits = p.dq_splits;
        const dim3 grid(static_cast<unsigned>(p.q_tiles), static_cast<unsigned>(a.kv * a.splits), z);
        if (p.few)
            hipLaunchKernelGGL((k_attend_dq<T, DP, 1, 4>), grid, dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((k_attend_dq<T, DP, 4, 1>), grid, dim3(kThreads), 0, s, a);
        if (a.splits > 1)
            hipLaunchKernelGGL((k_attend_reduce<T>),
                               dim3(static_cast<unsigned>(ceil_div(a.max_q * a.heads, 4)), z),
                               dim3(kThreads), 0, s, a, 0);
    }
    if (a.max_k > 0) {
        a.splits = p.dkv_splits;
        const dim3 grid(static_cast<unsigned>(p.k_tiles), static_cast<unsigned>(a.kv * a.splits), z);
        hipLaunchKernelGGL((k_attend_dkv<T, DP>), grid, dim3(kThreads), 0, s, a);
        if (a.splits > 1)
            hipLaunchKernelGGL((k_attend_reduce<T>),
                               dim3(static_cast<unsigned>(ceil_div(a.max_k * a.kv, 4)), z),
                               dim3(kThreads), 0, s, a, 1);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t run(const AttendArgs &a, const Plan &p, bool back, hipStream_t s) {
    if (a.d <= 64) return back ? backward<T, 64>(a, p, s) : forward<T, 64>(a, p, s);
    return back ? backward<T, 128>(a, p, s) : forward<T, 128>(a, p, s);
}

}  // namespace

size_t attend_bytes(const AttendArgs &a, bool backward) { return plan_for(a, backward).bytes; }

hipError_t launch_attend(AttendArgs a, bool backward, char *ws, hipStream_t s) {
    if (a.n_seq == 0 || (!backward && a.max_q == 0)) return hipSuccess;
    const Plan p = plan_for(a, backward);
    a.by_group = make_fastdiv(static_cast<uint32_t>(a.group));
    a.scale2 = a.scale * kLog2E;
    a.stat = reinterpret_cast<float2 *>(ws + p.stat);
    a.part_stat = reinterpret_cast<float2 *>(ws + p.part_stat);
    a.part = reinterpret_cast<float *>(ws + p.part);
    return a.type == GNN_F32 ? run<float>(a, p, backward, s) : run<bf16>(a, p, backward, s);
}

}  // namespace gnnmb
