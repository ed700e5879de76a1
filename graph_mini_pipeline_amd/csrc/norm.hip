// Layer norm over rows, and its backward pass.
//
// Forward, for a row x of d elements: m = sum x / d, v = sum (x - m)^2 / d, r = 1 / sqrt(v + eps),
// y = (x - m) r w + b.  The row stays in registers, so that v is summed of the differences themselves (the
// difference of two means loses all digits where m is large) and x is read once.
// Backward, with g = dy w and h = (x - m) r:
//   dx = r (g - sum g / d - h sum (g h) / d) (+ dres),  dw = sum over rows of dy h,  db = of dy.
// A lane group keeps its columns' sums of dw and db over all the rows it takes, a workgroup joins its
// groups', and the workgroups' are added by columns in their order: x and dy are read once, no atomics.
//
// A row is held by 8 to 64 lanes, or a workgroup, in pieces of eight elements; sums are fp32.
#include <type_traits>

#include "learn.hpp"

namespace gnnmb {

namespace {

constexpr int V = 8;
constexpr int kNormThreads = 256;

template <typename T>
__device__ __forceinline__ vec<float, V> load_piece(const T *p, int64_t left) {
    if (left >= V) return load_f32<T, V>(p);
    vec<float, V> v(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) v[i] = static_cast<float>(p[i]);
    return v;
}

template <typename T>
__device__ __forceinline__ void store_piece(T *p, int64_t left, vec<float, V> v) {
    if (left >= V) {
        store_f32<T, V>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) p[i] = static_cast<T>(v[i]);
}

__device__ __forceinline__ vec<float, V> load_param(const void *p, int32_t type, int64_t c, int64_t left, float otherwise) {
    if (p == nullptr) return vec<float, V>(otherwise);
    return type == GNN_BF16 ? load_piece(static_cast<const bf16 *>(p) + c, left)
                            : load_piece(static_cast<const float *>(p) + c, left);
}

__device__ __forceinline__ float sum_of(vec<float, V> v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
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

// G threads a row of up to G * V * CH elements.
template <typename TX, typename TO, int G, int CH>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void k_norm(NormArgs p) {
    constexpr int kThreads = G > kNormThreads ? G : kNormThreads, kRows = kThreads / G;
    __shared__ float lds[2][G > 64 ? G / 64 : 1];
    const int64_t n = load_count(p.d_n, p.n);
    const int l = threadIdx.x % G;
    const float d = static_cast<float>(p.d);      // divided by: equal elements have their own value as mean
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G; m < n; m += static_cast<int64_t>(gridDim.x) * kRows) {
        const TX *row = static_cast<const TX *>(p.x) + m * p.ld_x;
        vec<float, V> x[CH];
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t c = (j * G + l) * V;
            x[j] = load_piece(row + c, p.d - c);
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) s[0] += sum_of(x[j]);
        sum_row<G>(s, lds[0]);
        const float mean = s[0] / d;
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t left = p.d - (j * G + l) * V;
            x[j] -= mean;
            if (left < V) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i >= left) x[j][i] = 0.f;
            }
            s[0] += sum_of(x[j] * x[j]);
        }
        sum_row<G>(s, lds[1]);
        const float rstd = 1.f / sqrtf(s[0] / d + p.eps);
        if (l == 0) {
            if (p.mean) p.mean[m] = mean;
            if (p.rstd) p.rstd[m] = rstd;
        }
        TO *out = static_cast<TO *>(p.out) + m * p.ld_out;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t c = (j * G + l) * V, left = p.d - c;
            if (left <= 0) break;
            const vec<float, V> w = load_param(p.weight, p.param_type, c, left, 1.f);
            const vec<float, V> b = load_param(p.bias, p.param_type, c, left, 0.f);
            store_piece(out + c, left, x[j] * rstd * w + b);
        }
    }
}

template <typename TX, typename TO, int G, int CH>
__global__ __launch_bounds__(G > kNormThreads ? G : kNormThreads) void k_norm_backward(NormArgs p, float *sums) {
    constexpr int kThreads = G > kNormThreads ? G : kNormThreads, kRows = kThreads / G;
    constexpr int R = G > 512 ? 1 : 2;   // rows that a lane group loads at a time (128 registers a lane at G = 1024)
    __shared__ float lds[2][(G > 64 ? G / 64 : 1) * 2 * R];
    const int64_t n = load_count(p.d_n, p.n);
    const int l = threadIdx.x % G;
    const float inv_d = 1.f / static_cast<float>(p.d);
    vec<float, V> w[CH], dw[CH], db[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int64_t c = (j * G + l) * V;
        w[j] = load_param(p.weight, p.param_type, c, p.d - c, 1.f);
        dw[j] = db[j] = vec<float, V>(0.f);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int turn = 0;
    // (a workgroup that is one lane group leaves the loop as a whole)
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G; m0 < n; m0 += step * R, turn ^= 1) {
        vec<float, V> x[R][CH], g[R][CH];
        float s[2 * R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // past the end the last row again, which then counts for nothing
            const bool there = m0 + r * step < n;
            const int64_t m = there ? m0 + r * step : m0;
            const TX *row = static_cast<const TX *>(p.x) + m * p.ld_x;
            const TO *dy = static_cast<const TO *>(p.dout) + m * p.ld_dout;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int64_t c = (j * G + l) * V;
                x[r][j] = load_piece(row + c, p.d - c);
                g[r][j] = load_piece(dy + c, p.d - c);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = m0 + r * step < n;
            const int64_t m = there ? m0 + r * step : m0;
            const float mean = p.mean[m];
            rstd[r] = p.rstd[m];
            float sg = 0.f, sgh = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const vec<float, V> h = (x[r][j] - mean) * rstd[r];
                if (there) {
                    dw[j] += g[r][j] * h;
                    db[j] += g[r][j];
                }
                x[r][j] = h;
                g[r][j] *= w[j];
                sg += sum_of(g[r][j]);
                sgh += sum_of(g[r][j] * h);
            }
            s[2 * r] = sg;
            s[2 * r + 1] = sgh;
        }
        if (p.dx == nullptr) continue;
        sum_row<G>(s, lds[turn]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t m = m0 + r * step;
            if (m >= n) break;
            const float sg = s[2 * r] * inv_d, sgh = s[2 * r + 1] * inv_d;
            TX *dx = static_cast<TX *>(p.dx) + m * p.ld_dx;
            const TX *dres = p.dres ? static_cast<const TX *>(p.dres) + m * p.ld_dres : nullptr;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int64_t c = (j * G + l) * V, left = p.d - c;
                if (left <= 0) break;
                vec<float, V> v = (g[r][j] - sg - x[r][j] * sgh) * rstd[r];
                if (dres) v += load_piece(dres + c, left);
                store_piece(dx + c, left, v);
            }
        }
    }
    if (sums == nullptr) return;
    // the groups' sums, joined; part b: [dweight, dbias] of d columns each
    float *to = sums + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
    if (kRows == 1) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int64_t c = (j * G + l) * V, left = p.d - c;
            if (left <= 0) break;
            store_piece(to + c, left, dw[j]);
            store_piece(to + p.d + c, left, db[j]);
        }
        return;
    }
    __shared__ float joined[kRows > 1 ? kRows * G * V * CH : 1];
    constexpr int kWide = G * V * CH;
    for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) joined[threadIdx.x / G * kWide + (j * G + l) * V + i] = half ? db[j][i] : dw[j][i];
        __syncthreads();
        for (int c = threadIdx.x; c < p.d; c += kThreads) {
            float v = 0.f;
            for (int r = 0; r < kRows; ++r) v += joined[r * kWide + c];
            to[half * p.d + c] = v;
        }
    }
}

// Threads a row, and pieces a thread: f(G, CH).
template <typename F>
hipError_t by_forward_width(int64_t d, F f) {
    using std::integral_constant;
    const integral_constant<int, 8> g8{};
    const integral_constant<int, 16> g16{};
    const integral_constant<int, 32> g32{};
    const integral_constant<int, 64> g64{};
    const integral_constant<int, 256> g256{};
    const integral_constant<int, 1> c1{};
    const integral_constant<int, 2> c2{};
    const integral_constant<int, 4> c4{};
    const integral_constant<int, 8> c8{};
    if (d <= 8 * V) return f(g8, c1);
    if (d <= 16 * V) return f(g16, c1);
    if (d <= 32 * V) return f(g32, c1);
    if (d <= 64 * V) return f(g64, c1);
    if (d <= 128 * V) return f(g64, c2);
    if (d <= 256 * V) return f(g64, c4);
    if (d <= 512 * V) return f(g64, c8);
    if (d <= 1024 * V) return f(g256, c4);
    return f(g256, c8);
}

// Fewer pieces a thread: it keeps the sums of dw and db beside x and dy.
template <typename F>
hipError_t by_backward_width(int64_t d, F f) {
    using std::integral_constant;
    const integral_constant<int, 8> g8{};
    const integral_constant<int, 16> g16{};
    const integral_constant<int, 32> g32{};
    const integral_constant<int, 64> g64{};
    const integral_constant<int, 256> g256{};
    const integral_constant<int, 512> g512{};
    const integral_constant<int, 1024> g1024{};
    const integral_constant<int, 1> c1{};
    const integral_constant<int, 2> c2{};
    if (d <= 8 * V) return f(g8, c1);
    if (d <= 16 * V) return f(g16, c1);
    if (d <= 32 * V) return f(g32, c1);
    if (d <= 64 * V) return f(g64, c1);
    if (d <= 128 * V) return f(g64, c2);
    if (d <= 256 * V) return f(g256, c1);
    if (d <= 512 * V) return f(g256, c2);
    if (d <= 1024 * V) return f(g512, c2);
    return f(g1024, c2);
}

// Workgroups of the backward pass: as many as keep memory busy, and no more than their partial sums are
// worth (two a compute unit for wide rows: 512 x 2 x 4096 sums take 3% of the time of 32768 rows).
int64_t backward_blocks(int64_t n, int64_t d) {
    const int64_t rows = d <= 128 * V ? kNormThreads / (d <= 8 * V ? 8 : d <= 16 * V ? 16 : d <= 32 * V ? 32 : 64) : 1;
    int64_t blocks = (n + rows * 2 - 1) / (rows * 2);
    const int64_t most = d > 128 * V ? 512 : 1024;
    if (blocks > most) blocks = most;
    return blocks < 1 ? 1 : blocks;
}

template <typename TX, typename TO>
hipError_t norm(const NormArgs &a, hipStream_t s) {
    return by_forward_width(a.d, [&](auto g, auto ch) {
        constexpr int G = g, CH = ch, kThreads = G > kNormThreads ? G : kNormThreads;
        int64_t blocks = (a.n + kThreads / G - 1) / (kThreads / G);
        if (blocks > 1 << 20) blocks = 1 << 20;
        k_norm<TX, TO, G, CH><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
        return hipGetLastError();
    });
}

template <typename TX, typename TO>
hipError_t norm_backward(const NormArgs &a, hipStream_t s) {
    const int64_t blocks = backward_blocks(a.n, a.d);
    float *sums = a.dweight || a.dbias ? reinterpret_cast<float *>(a.ws) : nullptr;
    const hipError_t err = by_backward_width(a.d, [&](auto g, auto ch) {
        constexpr int G = g, CH = ch, kThreads = G > kNormThreads ? G : kNormThreads;
        k_norm_backward<TX, TO, G, CH><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, sums);
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
