// Layer norm over rows, and its backward pass.
//
// Forward, for a row x of d elements: m = sum x / d, v = sum (x - m)^2 / d, r = 1 / sqrt(v + eps),
// y = (x - m) r w + b.  The row stays in registers, so that v is summed of the differences themselves (the
// difference of two means loses all digits where m is large) and x is read once.  m as it is first summed is off by
// some roundings of the row's size: with it alone a row of 768 times 12345.678 had results of 0.3 for 0.  The
// differences, exact where m is large beside them, have the mean c = sum (x - m) / d by which m is put right:
//   y = (x - m - c) r w + b,  v = sum (x - m)^2 / d - c^2,  and m + c is the mean,
// where m^2 > 4 v; of smaller means the differences' roundings are the larger ones (32768 x 4096 bf16 with means of a
// fiftieth of their spread: these are 4e-8 off, 9e-7 if they were put right, too), and c is 0.
// (180224 x 100 fp32 19.8 us for 19.1, 32768 x 4096 bf16 110.1 for 109.6, 8192 x 8192 50.5 for 48.0.)
// Backward, with g = dy w and h = (x - m) r:
//   dx = r (g - sum g / d - h sum (g h) / d) (+ dres),  dw = sum over rows of dy h,  db = of dy.
// A lane group keeps its columns' sums of dw and db over all the rows it takes, a workgroup joins its
// groups', and the workgroups' are added by columns in their order: x and dy are read once, no atomics.
//
// A row is held by 8 to 64 lanes, or a workgroup, in pieces of eight elements; sums are fp32.  Up to 4096
// elements a lane has at most two pieces of a row and takes two rows at a time: few enough registers for
// the loads of several workgroups to be under way on a compute unit.
//
// What bounds it: memory.  32768 x 4096 bf16: forward 106 us (5.1 TB/s), backward with a residual gradient
// 212 (5.2 TB/s), its columns' join 5; 180224 x 100 fp32 to bf16: 25, 40 and 5.  (One wavefront a row with eight
// pieces a lane took 214 us forward, rows kept in fp32 between the passes 316 backward.)  Rows over 8192 elements
// fill the registers of a compute unit one at a time, and the backward pass spills half of a lane's 128 (132 to 184 bytes of
// scratch): 8000 x 16384 3.4 TB/s in fp32, 2.6 in bf16.  A single row of 4096: 4 us, launch and four dependent turns.
#include <type_traits>

#include "learn.hpp"

namespace gnnmb {

namespace {

constexpr int kNormThreads = 256;

// Piece j of lane l of G: V elements, the row's last ones where it would reach past its end.  Those that
// an earlier piece holds too (the first `twice`) count once in sums; computed and stored they are the same.
template <int G, int V>
struct Piece {
    int c;           // first column
    int twice;       // V or more: the piece is a copy altogether
    __device__ __forceinline__ Piece(int j, int l, int cols) {
        const int at = (j * G + l) * V;
        c = at < cols - V ? at : cols - V;
        twice = at - c;
    }
    // The elements that count, zeros for others; `ragged` (uniform): some piece of the row counts in part.
    __device__ __forceinline__ vec<float, V> counted(vec<float, V> v, bool ragged) const {
        if (ragged) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i >= twice ? v[i] : 0.f;
        }
        return v;
    }
    __device__ __forceinline__ float sum(vec<float, V> v, bool ragged) const { return sum(counted(v, ragged)); }
    __device__ __forceinline__ float sum(vec<float, V> v) const {
        float s = v[0];
        if constexpr (V == 8) s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        return twice < V ? s : 0.f;
    }
};

template <int V, typename T>
__device__ __forceinline__ vec<T, V> load_raw(const T *p) {
    return *reinterpret_cast<const typename loose<T, V>::type *>(p);
}

// Forgets what has been computed of v: what a later pass needs of it is computed again from the piece as
// it was loaded (half the registers for bf16), not kept.
template <typename T, int V>
__device__ __forceinline__ void again(vec<T, V> &v) {
    if constexpr (sizeof(T) * V == 16) {
        typedef vec<uint32_t, 4> Words;
        Words x = __builtin_bit_cast(Words, v);
        asm volatile("" : "+v"(x));
        v = __builtin_bit_cast(vec<T, V>, x);
    }
}

template <int V>
__device__ __forceinline__ vec<float, V> load_param(const void *p, int32_t type, int c, float otherwise) {
    if (p == nullptr) return vec<float, V>(otherwise);
    return type == GNN_BF16 ? load_f32<bf16, V>(static_cast<const bf16 *>(p) + c)
                            : load_f32<float, V>(static_cast<const float *>(p) + c);
}

// The sums of N values over the G threads of a row, in all of them.  G over 64: `lds` has N floats a
// wavefront, which the next call must not use (two buffers in turn need one barrier a call).
template <int G, int N>
__device__ __forceinline__ void sum_row(float (&v)[N], float *lds) {
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, 64);
    if (G <= 64) return;
    constexpr int kWaves = G / 64;
    const int w = threadIdx.x / 64;
    if (lane_id() == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) lds[w * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kWaves; ++j) s += lds[j * N + i];
        v[i] = s;
    }
}

// Which of the workgroup's rows this thread works on: one for a wavefront of lane groups of 64 or more.
template <int G>
__device__ __forceinline__ int group_of() {
    const int g = static_cast<int>(threadIdx.x) / G;
    return G >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// G threads a row of up to G * V * CH elements, R rows at a time; the parameters stay in registers.
template <typename TX, typename TO, int G, int CH, int R, int V>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void k_norm(NormArgs p) {
    constexpr int kThreads = G > kNormThreads ? G : kNormThreads, kRows = kThreads / G;
    typedef vec<float, V> Wide;
    __shared__ float lds[2][(G > 64 ? G / 64 : 1) * 2 * R];
    const int64_t n = load_count(p.d_n, p.n);
    const int l = threadIdx.x % G, cols = static_cast<int>(p.d);
    const bool ragged = cols % V != 0;
    const float d = static_cast<float>(p.d), inv_d = 1.f / d;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    Wide w[CH], b[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const Piece<G, V> at(j, l, cols);
        w[j] = load_param<V>(p.weight, p.param_type, at.c, 1.f);
        b[j] = load_param<V>(p.bias, p.param_type, at.c, 0.f);
    }
    // (a workgroup that is one lane group leaves the loop as a whole)
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + group_of<G>(); m0 < n; m0 += step * R) {
        vec<TX, V> raw[R][CH];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // past the end the first row again, which is not stored
            const int64_t m = m0 + r * step < n ? m0 + r * step : m0;
            const TX *row = static_cast<const TX *>(p.x) + m * p.ld_x;
#pragma unroll
            for (int j = 0; j < CH; ++j) raw[r][j] = load_raw<V>(row + Piece<G, V>(j, l, cols).c);
        }
        float s[R], e[2 * R], mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j)
                s[r] += Piece<G, V>(j, l, cols).sum(__builtin_convertvector(raw[r][j], Wide), ragged);
        }
        sum_row<G>(s, lds[0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = s[r] / d;      // (as a product it would be fused into the subtraction, whose m is then another)
            e[2 * r] = e[2 * r + 1] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                again(raw[r][j]);
                const Piece<G, V> at(j, l, cols);
                const Wide x = at.counted(__builtin_convertvector(raw[r][j], Wide) - mean[r], ragged);
                e[2 * r] += at.sum(x);
                e[2 * r + 1] += at.sum(x * x);
            }
        }
        sum_row<G>(e, lds[1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t m = m0 + r * step;
            if (m >= n) break;
            float v = e[2 * r + 1] * inv_d;
            const float c = mean[r] * mean[r] > 4.f * v ? e[2 * r] / d : 0.f;
            v -= c * c;
            if (v < 0.f) v = 0.f;                     // (a NaN stays)
            const float rstd = 1.f / sqrtf(v + p.eps);
            if (l == 0) {
                if (p.mean) p.mean[m] = mean[r] + c;
                if (p.rstd) p.rstd[m] = rstd;
            }
            TO *out = static_cast<TO *>(p.out) + m * p.ld_out;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const Piece<G, V> at(j, l, cols);
                again(raw[r][j]);
                if (at.twice < V)
                    store_f32<TO, V>(out + at.c, (__builtin_convertvector(raw[r][j], Wide) - mean[r] - c) * rstd * w[j] + b[j]);
            }
        }
    }
}

template <typename TX, typename TO, int G, int CH, int R, int V>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void k_norm_backward(NormArgs p, float *sums) {
    constexpr int kThreads = G > kNormThreads ? G : kNormThreads, kRows = kThreads / G;
    typedef vec<float, V> Wide;
    __shared__ float lds[2][(G > 64 ? G / 64 : 1) * 2 * R];
    const int64_t n = load_count(p.d_n, p.n);
    const int l = threadIdx.x % G, cols = static_cast<int>(p.d);
    const bool ragged = cols % V != 0;
    const float inv_d = 1.f / static_cast<float>(p.d);
    Wide w[CH], dw[CH], db[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        w[j] = load_param<V>(p.weight, p.param_type, Piece<G, V>(j, l, cols).c, 1.f);
        dw[j] = db[j] = Wide(0.f);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int turn = 0;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + group_of<G>(); m0 < n; m0 += step * R, turn ^= 1) {
        vec<TX, V> x[R][CH], dres[R][CH];
        vec<TO, V> dy[R][CH];
        float s[2 * R], mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // past the end the first row again, which then counts for nothing
            const int64_t m = m0 + r * step < n ? m0 + r * step : m0;
            const TX *row = static_cast<const TX *>(p.x) + m * p.ld_x;
            const TO *from = static_cast<const TO *>(p.dout) + m * p.ld_dout;
            mean[r] = p.mean[m];
            rstd[r] = p.rstd[m];
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = Piece<G, V>(j, l, cols).c;
                x[r][j] = load_raw<V>(row + c);
                dy[r][j] = load_raw<V>(from + c);
                if (p.dres) dres[r][j] = load_raw<V>(static_cast<const TX *>(p.dres) + m * p.ld_dres + c);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = r == 0 || m0 + r * step < n;
            s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const Piece<G, V> at(j, l, cols);
                const Wide h = (__builtin_convertvector(x[r][j], Wide) - mean[r]) * rstd[r];
                const Wide g = __builtin_convertvector(dy[r][j], Wide);
                if (there) {
                    dw[j] += g * h;
                    db[j] += g;
                }
                const Wide gw = g * w[j];
                s[2 * r] += at.sum(gw, ragged);
                s[2 * r + 1] += at.sum(gw * h, ragged);
            }
        }
        if (p.dx == nullptr) continue;
        sum_row<G>(s, lds[turn]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t m = m0 + r * step;
            if (m >= n) break;
            const float sg = s[2 * r] * inv_d, sgh = s[2 * r + 1] * inv_d;
            TX *dx = static_cast<TX *>(p.dx) + m * p.ld_dx;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const Piece<G, V> at(j, l, cols);
                if (at.twice >= V) continue;
                again(x[r][j]);
                again(dy[r][j]);
                const Wide h = (__builtin_convertvector(x[r][j], Wide) - mean[r]) * rstd[r];
                Wide v = (__builtin_convertvector(dy[r][j], Wide) * w[j] - sg - h * sgh) * rstd[r];
                if (p.dres) v += __builtin_convertvector(dres[r][j], Wide);
                store_f32<TX, V>(dx + at.c, v);
            }
        }
    }
    if (sums == nullptr) return;
    // the groups' sums, joined: [dweight, dbias] of the workgroup
    float *to = sums + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
    if (kRows == 1) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const Piece<G, V> at(j, l, cols);
            if (at.twice >= V) continue;
            store_f32<float, V>(to + at.c, dw[j]);
            store_f32<float, V>(to + p.d + at.c, db[j]);
        }
        return;
    }
    constexpr int kWide = G * V * CH;
    __shared__ float joined[kRows > 1 ? kRows * kWide : 1];
    for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const Piece<G, V> at(j, l, cols);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at.twice < V) joined[threadIdx.x / G * kWide + at.c + i] = half ? db[j][i] : dw[j][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += kThreads) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += joined[r * kWide + c];
            to[half * p.d + c] = v;
        }
    }
}

// Threads a row, pieces a thread and rows at a time, and elements a piece, by the row's width: f(G, CH, R, V).
template <typename F>
hipError_t by_width(int64_t d, F f) {
    using std::integral_constant;
    const integral_constant<int, 1> one{};
    const integral_constant<int, 2> two{};
    const integral_constant<int, 8> eight{};
    if (d < 8) return f(eight, one, two, one);
    if (d <= 64) return f(eight, one, two, eight);
    if (d <= 128) return f(integral_constant<int, 16>{}, one, two, eight);
    if (d <= 256) return f(integral_constant<int, 32>{}, one, two, eight);
    if (d <= 512) return f(integral_constant<int, 64>{}, one, two, eight);
    if (d <= 1024) return f(integral_constant<int, 64>{}, two, two, eight);
    if (d <= 2048) return f(integral_constant<int, 256>{}, one, two, eight);
    if (d <= 4096) return f(integral_constant<int, 256>{}, two, two, eight);
    if (d <= 8192) return f(integral_constant<int, 512>{}, two, two, eight);
    return f(integral_constant<int, 1024>{}, two, one, eight);      // 128 registers a lane
}

int64_t row_blocks(int64_t n, int g, int r, int64_t most) {
    const int rows = g < kNormThreads ? kNormThreads / g : 1;
    int64_t blocks = (n + rows * r - 1) / (rows * r);
    if (blocks > most) blocks = most;
    return blocks < 1 ? 1 : blocks;
}

// Workgroups of the backward pass: one for each turn of its rows, up to as many as keep memory busy.  Each leaves 8 d
// bytes of sums, a small part of what thousands of rows take; of some hundred wide rows, it is as much again as the
// rows themselves (512 x 16384 bf16 53 us, 1 TB/s of x, dout and dx, where 8000 rows run at 2.6).
int64_t backward_blocks(int64_t n, int64_t d) {
    int64_t blocks = 0;
    (void)by_width(d, [&](auto g, auto, auto r, auto) {
        blocks = row_blocks(n, g, r, d > 1024 ? 512 : 1024);
        return hipSuccess;
    });
    return blocks;
}

template <typename TX, typename TO>
hipError_t norm(const NormArgs &a, hipStream_t s) {
    return by_width(a.d, [&](auto g, auto ch, auto r, auto v) {
        constexpr int G = g, CH = ch, R = r, V = v, kThreads = G > kNormThreads ? G : kNormThreads;
        k_norm<TX, TO, G, CH, R, V><<<static_cast<unsigned>(row_blocks(a.n, G, R, 2048)), kThreads, 0, s>>>(a);
        return hipGetLastError();
    });
}

template <typename TX, typename TO>
hipError_t norm_backward(const NormArgs &a, hipStream_t s) {
    const int64_t blocks = backward_blocks(a.n, a.d);
    float *sums = a.dweight || a.dbias ? reinterpret_cast<float *>(a.ws) : nullptr;
    const hipError_t err = by_width(a.d, [&](auto g, auto ch, auto r, auto v) {
        constexpr int G = g, CH = ch, R = r, V = v, kThreads = G > kNormThreads ? G : kNormThreads;
        k_norm_backward<TX, TO, G, CH, R, V><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, sums);
        return hipGetLastError();
    });
    if (err != hipSuccess || sums == nullptr) return err;
    return launch_column_sums(sums, 2 * a.d, static_cast<int>(blocks), a.d, a.d, a.param_type, a.dweight, a.dbias, s);
}

}  // namespace

size_t norm_bytes(int64_t n, int64_t d) {
    return static_cast<size_t>(backward_blocks(n, d)) * 2 * static_cast<size_t>(d) * sizeof(float);
}

hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    if (a.x_type == GNN_BF16) return a.out_type == GNN_BF16 ? norm<bf16, bf16>(a, s) : norm<bf16, float>(a, s);
    return a.out_type == GNN_BF16 ? norm<float, bf16>(a, s) : norm<float, float>(a, s);
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s) {
    if (a.x_type == GNN_BF16)
        return a.out_type == GNN_BF16 ? norm_backward<bf16, bf16>(a, s) : norm_backward<bf16, float>(a, s);
    return a.out_type == GNN_BF16 ? norm_backward<float, bf16>(a, s) : norm_backward<float, float>(a, s);
}

}  // namespace gnnmb
