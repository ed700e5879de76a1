// Dense layers on the matrix cores: y = act(x W + b) + r, the gated pair y = act(x Wg + bg) (x Wu + bu),
// and their gradients.
//
// Forward is one product with its epilogue (dense.hpp); a gated layer's two products share the tiles of x
// and meet in the epilogue's registers.  Backward, with z kept by the forward pass:
//   dz = dy act'(z)                 (k_slopes; gated: dg = dy u act'(g), du = dy act(g))
//   db = the sums of dz's columns   (partial sums by k_slopes, k_column_sums)
//   dx = dz W^T, dW = x^T dz        (gated: dx = dg Wg^T + du Wu^T in one product over two segments)
// Without an activation dz is dy itself.
//
// Numbers.  Products are summed in fp32: bf16 on the 16-bit matrix instructions, fp32 on the fp32 ones.
// The dz of a bf16 layer is rounded to bf16 for its products, an error of the size of the result's own
// rounding where few terms are summed and below it where many are; a sum of fewer than kShortSum terms
// takes dz in two planes, its bf16 and the bf16 of what that leaves.  No atomic touches a sum: the parts
// of a split sum are added in their order.
#include "dense.hpp"

namespace gnnmb {

namespace {

// out[c] = the sum of `parts` rows of sums; a workgroup takes 32 columns, 32 rows at a time.
constexpr int kColumnHigh = 32;
template <typename T>
__global__ __launch_bounds__(32 * kColumnHigh) void k_column_sums(const float *sums, int64_t ld, int parts, int64_t cols,
                                                                  int64_t second, void *out0, void *out1) {
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t c = blockIdx.x * 32ll + x;
    T *out = static_cast<T *>(blockIdx.y ? out1 : out0);
    if (out == nullptr) return;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int i = y; i < parts; i += kColumnHigh) s += sums[i * ld + blockIdx.y * second + c];
    }
    __shared__ float lds[kColumnHigh][33];
    lds[y][x] = s;
    __syncthreads();
    if (y == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < kColumnHigh; ++i) s += lds[i][x];
        out[c] = static_cast<T>(s);
    }
}

constexpr int kCus = 256;

// ---- splits of a summed length, joined -----------------------------------------------------------------

template <typename T, bool PAIR>
__global__ __launch_bounds__(256) void k_product_join(ProductArgs p, int rows_are_n, int wide_log2) {
    const int64_t rows = rows_are_n ? load_count(p.d_n, p.rows) : p.rows;
    const int wide = 1 << wide_log2;
    const int z = blockIdx.y;
    const int64_t n = ((static_cast<int64_t>(blockIdx.z) << wide_log2) + (threadIdx.x & (wide - 1))) * 4;
    if (n >= p.cols) return;
    const int64_t step = gridDim.x * static_cast<int64_t>(256 >> wide_log2);
    const int64_t products = PAIR ? 2 : p.products;
    for (int64_t m = blockIdx.x * static_cast<int64_t>(256 >> wide_log2) + (threadIdx.x >> wide_log2); m < rows; m += step) {
        vec<float, 4> v(0.f), u(0.f);
        const float *from = p.part + (z * p.rows + m) * p.ld_part + n;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            v += *reinterpret_cast<const vec<float, 4> *>(from);
            if (PAIR) u += *reinterpret_cast<const vec<float, 4> *>(from + p.rows * p.ld_part);
            from += products * p.rows * p.ld_part;
        }
        finish<T, 4, PAIR>(p.e, z, m, n, p.cols - n, v, u);
    }
}

template <typename T>
hipError_t launch_join(const ProductArgs &a, bool rows_are_n, bool pair, hipStream_t s) {
    int wide = 0;
    while (wide < 8 && (4 << wide) < a.cols) ++wide;
    const int64_t high = 256 >> wide, groups = (a.cols + (4 << wide) - 1) / (4 << wide);
    int64_t blocks = (a.rows + high - 1) / high;
    if (blocks > 4096) blocks = 4096;
    const dim3 grid(static_cast<unsigned>(blocks), pair ? 1 : a.products, static_cast<unsigned>(groups));
    if (pair)
        k_product_join<T, true><<<grid, 256, 0, s>>>(a, rows_are_n, wide);
    else
        k_product_join<T, false><<<grid, 256, 0, s>>>(a, rows_are_n, wide);
    return hipGetLastError();
}

// ---- planning ------------------------------------------------------------------------------------------

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether the product's operands can go into LDS directly: whole 16-byte pieces everywhere.
bool direct_fits(const ProductArgs &a, int form, bool pair, int size) {
    const int64_t elems = 16 / size;
    const int segs = a.segs > a.short_segs ? a.segs : a.short_segs;
    bool fits = a.ld_a % elems == 0 && a.ld_b % elems == 0;
    for (int i = 0; i < segs; ++i) {
        fits = fits && aligned16(a.a[i]);
        for (int z = 0; z < (pair ? 2 : a.products); ++z) fits = fits && aligned16(a.b[z][i]);
    }
    if (form == kGradW) fits = fits && a.rows % elems == 0;
    if (form != kGradX) fits = fits && a.cols % elems == 0;
    return fits;
}

struct Tiling {
    int tile;
    int64_t splits;
};

// The tile and the number of parts of the summed length with the least time by a model: each compute unit
// works off its share of the workgroups, a workgroup takes `step` us for 128 bytes of the summed length
// when it has the unit to itself with as many others as fit (and at least `alone`), and a split sum goes
// through memory once more.
Tiling choose_tiling(int form, int type, bool pair, bool direct, int64_t rows, int64_t cols, int64_t k, int segs, int products) {
    const bool bf = type == GNN_BF16;
    const int64_t bk = bf ? 64 : 32;
    const int64_t steps = (k + bk - 1) / bk * segs;
    Tiling best{kTile128, 1};
    double least = 1e30;
    for (int tile = kTile256; tile <= kTile32; ++tile) {
        if (tile == kTile256 && (!bf || !direct)) continue;
        if (tile == kTile32 && (form == kGradW || rows > 64)) continue;
        // few rows: a gated pair is taken as two products whose parts are joined
        const bool paired = pair && tile != kTile32;
        const int64_t tr = tile_rows(tile), tc = tile_cols(tile, paired);
        const int64_t tiles = ((rows + tr - 1) / tr) * ((cols + tc - 1) / tc) * (tile == kTile32 && pair ? 2 : products);
        const double step = tile == kTile256 ? 1.9 : tile == kTile128 ? (bf ? 0.65 : 2.0) : (bf ? 0.5 : 0.6);
        const double alone = tile == kTile256 ? 1.9 : tile == kTile128 ? (bf ? 0.8 : 2.0) : 0.6;
        for (int64_t splits = 1; splits <= 64 && splits <= (steps > 0 ? steps : 1); splits += splits < 8 ? 1 : splits / 4) {
            const bool joined = splits > 1 || (tile == kTile32 && pair);
            const int64_t each = (steps + splits - 1) / splits;
            const int64_t load = (tiles * splits + kCus - 1) / kCus;
            double us = load * (each * step + 1.0);
            const double one = each * alone + 2.0;
            if (us < one) us = one;
            if (joined) us += 4.0 + splits * products * (pair ? 2 : 1) * rows * cols * 8e-6 / 3.0;
            if (us < least) {
                least = us;
                best = {tile, splits};
            }
        }
    }
    return best;
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Floats of the parts that a product's plan needs.
int64_t part_floats(const Tiling &t, bool pair, int64_t rows, int64_t cols, int products) {
    const bool joined = t.splits > 1 || (t.tile == kTile32 && pair);
    return joined ? t.splits * (pair ? 2 : products) * rows * round_up(cols, 4) : 0;
}

// Whatever the operands' alignment.
int64_t most_part_floats(int form, int type, bool pair, int64_t rows, int64_t cols, int64_t k, int segs, int products) {
    int64_t most = 0;
    for (int direct = 0; direct < 2; ++direct) {
        const int64_t f = part_floats(choose_tiling(form, type, pair, direct, rows, cols, k, segs, products), pair, rows, cols, products);
        most = f > most ? f : most;
    }
    return most;
}

// What a product needs beside its operands: where parts of its sum go (ws).
hipError_t product(ProductArgs a, int form, int type, bool pair, char *ws, hipStream_t s) {
    const bool direct = direct_fits(a, form, pair, type == GNN_BF16 ? 2 : 4);
    const Tiling t = choose_tiling(form, type, pair, direct, a.rows, a.cols, a.k, a.segs, a.products);
    const bool joined = t.splits > 1 || (t.tile == kTile32 && pair);
    a.splits = static_cast<int32_t>(t.splits);
    a.part = joined ? reinterpret_cast<float *>(ws) : nullptr;
    a.ld_part = round_up(a.cols, 4);
    ProductArgs b = a;
    if (t.tile == kTile32 && pair) b.products = 2;
    const ProductPlan plan{form, t.tile, pair && t.tile != kTile32, direct};
    const hipError_t err = type == GNN_BF16 ? launch_product_bf16(b, plan, s) : launch_product_f32(b, plan, s);
    if (err != hipSuccess || !joined) return err;
    return type == GNN_BF16 ? launch_join<bf16>(a, form != kGradW, pair, s) : launch_join<float>(a, form != kGradW, pair, s);
}

// ---- the gradient of the sums ----------------------------------------------------------------------------

struct SlopeArgs {
    const void *dout, *pre[2];
    int64_t ld_dout, ld_pre;
    const int64_t *d_n;
    int64_t n, cols;
    int32_t act, store;          // store = 0: dz is dout, only its columns are summed
    int32_t planes_wide;         // two planes of every row (else of fewer than kShortSum rows)
    void *dz, *rest;             // [n, ld_dz] each; the other projection's columns start at `second`
    int64_t ld_dz, second;
    float *sums;                 // [gridDim.y][ld_sums], NULL: none
    int64_t ld_sums;
};

constexpr int kSlopeWide = 32, kSlopeHigh = 8;     // threads of a workgroup
constexpr int kSlopeBlocks = 2048;                 // workgroups at most, unless the columns alone need more
constexpr int kSlopeRows = 4;                      // rows that a thread loads at a time

template <typename T, bool PAIR>
__global__ __launch_bounds__(kSlopeWide * kSlopeHigh) void k_slopes(SlopeArgs p) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    constexpr bool kFast = sizeof(T) == 2;
    const int64_t n = load_count(p.d_n, p.n);
    const bool planes = kFast && (p.planes_wide || n < kShortSum);
    const int x = threadIdx.x % kSlopeWide, y = threadIdx.x / kSlopeWide;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * kSlopeWide + x) * V, left = p.cols - c;
    vec<float, V> sum0(0.f), sum1(0.f);
    const int64_t step = static_cast<int64_t>(gridDim.y) * kSlopeHigh;
    const auto keep = [&](int64_t at, vec<float, V> v) {
        T *to = static_cast<T *>(p.dz) + at;
        const vec<T, V> r = __builtin_convertvector(v, vec<T, V>);
        // dz is the library's own and its lines are padded
        *reinterpret_cast<vec<T, V> *>(to) = r;
        if (planes) {
            v -= __builtin_convertvector(r, vec<float, V>);
            *reinterpret_cast<vec<T, V> *>(static_cast<T *>(p.rest) + at) = __builtin_convertvector(v, vec<T, V>);
        }
    };
    if (left > 0) {
        for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kSlopeHigh + y; m0 < n; m0 += step * kSlopeRows) {
            vec<float, V> d[kSlopeRows], a[kSlopeRows], b[kSlopeRows];
#pragma unroll
            for (int i = 0; i < kSlopeRows; ++i) {
                const int64_t m = m0 + i * step;
                if (m >= n) break;
                d[i] = load_some<T, V>(static_cast<const T *>(p.dout) + m * p.ld_dout + c, left);
                if (p.store) a[i] = load_some<T, V>(static_cast<const T *>(p.pre[0]) + m * p.ld_pre + c, left);
                if (PAIR) b[i] = load_some<T, V>(static_cast<const T *>(p.pre[1]) + m * p.ld_pre + c, left);
            }
#pragma unroll
            for (int i = 0; i < kSlopeRows; ++i) {
                const int64_t m = m0 + i * step;
                if (m >= n) break;
                vec<float, V> g = d[i];
                if (p.store) {
                    const vec<float, V> slope = activate_slope<kFast, V>(p.act, a[i]);
                    g = PAIR ? g * b[i] * slope : g * slope;
                    keep(m * p.ld_dz + c, g);
                    if (PAIR) {
                        const vec<float, V> u = d[i] * a[i];
                        keep(m * p.ld_dz + p.second + c, u);
                        sum1 += u;
                    }
                }
                sum0 += g;
            }
        }
    }
    if (p.sums == nullptr) return;
    __shared__ float lds[kSlopeHigh][(PAIR ? 2 : 1) * V][kSlopeWide + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        lds[y][i][x] = sum0[i];
        if (PAIR) lds[y][V + i][x] = sum1[i];
    }
    __syncthreads();
    for (int e = y; e < (PAIR ? 2 : 1) * V; e += kSlopeHigh) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSlopeHigh; ++i) s += lds[i][e][x];
        if (e % V < left) p.sums[blockIdx.y * p.ld_sums + (e >= V ? p.second : 0) + c + e % V] = s;
    }
}

int slope_parts(int64_t n, int64_t cols, int type) {
    const int64_t wide = kSlopeWide * (type == GNN_BF16 ? 8 : 4);
    const int64_t across = (cols + wide - 1) / wide;
    int64_t parts = (n + kSlopeHigh * kSlopeRows - 1) / (kSlopeHigh * kSlopeRows);
    const int64_t most = kSlopeBlocks / across;
    if (parts > most) parts = most;
    return static_cast<int>(parts < 1 ? 1 : parts);
}

// ---- workspace -----------------------------------------------------------------------------------------

struct DenseSpace {
    char *dz, *rest, *sums, *part;
    int64_t ld_dz, second;
    bool wide;               // two planes of every row: dx sums few terms
    size_t bytes;
};

// dz has whole 128-byte lines; of its second plane only what a short sum reads is there.
DenseSpace carve_dense(const DenseArgs &a, char *ws) {
    DenseSpace w{};
    const int mats = a.pair ? 2 : 1;
    const int64_t size = a.type == GNN_BF16 ? 2 : 4;
    w.second = round_up(a.d_out, 128 / size);
    w.ld_dz = w.second * mats;
    w.wide = a.type == GNN_BF16 && a.d_out * mats < kShortSum;
    size_t at = 0;
    const auto take = [&](char **p, int64_t bytes) {
        *p = ws + at;
        at += static_cast<size_t>(round_up(bytes < 1 ? 1 : bytes, 256));
    };
    take(&w.dz, a.n * w.ld_dz * size);
    const int64_t rest_rows = a.type != GNN_BF16 ? 0 : w.wide || a.n < kShortSum ? a.n : kShortSum;
    take(&w.rest, rest_rows * w.ld_dz * size);
    take(&w.sums, static_cast<int64_t>(slope_parts(a.n, a.d_out, a.type)) * w.ld_dz * 4);
    int64_t floats = 0;
    for (int i = 1; i <= 2; ++i) {     // one plane or two, one weight's gradient or two
        const int64_t dx = most_part_floats(kGradX, a.type, false, a.n, a.d_in, a.d_out, i * mats, 1);
        const int64_t dw = most_part_floats(kGradW, a.type, false, a.d_in, a.d_out, a.n, 1, i < mats ? i : mats);
        floats = dx > floats ? dx : floats;
        floats = dw > floats ? dw : floats;
    }
    take(&w.part, 4 * floats);
    w.bytes = at;
    return w;
}

template <typename T>
hipError_t launch_slopes(const SlopeArgs &a, bool pair, hipStream_t s) {
    const int64_t wide = kSlopeWide * 16 / static_cast<int64_t>(sizeof(T));
    const dim3 grid(static_cast<unsigned>((a.cols + wide - 1) / wide),
                    slope_parts(a.n, a.cols, sizeof(T) == 2 ? GNN_BF16 : GNN_F32));
    if (pair)
        k_slopes<T, true><<<grid, kSlopeWide * kSlopeHigh, 0, s>>>(a);
    else
        k_slopes<T, false><<<grid, kSlopeWide * kSlopeHigh, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_column_sums(const float *sums, int64_t ld, int parts, int64_t cols, int64_t second, int type, void *out0,
                              void *out1, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>((cols + 31) / 32), 2);
    if (type == GNN_BF16)
        k_column_sums<bf16><<<grid, 32 * kColumnHigh, 0, s>>>(sums, ld, parts, cols, second, out0, out1);
    else
        k_column_sums<float><<<grid, 32 * kColumnHigh, 0, s>>>(sums, ld, parts, cols, second, out0, out1);
    return hipGetLastError();
}

size_t dense_bytes(const DenseArgs &a, bool backward) {
    if (backward) return carve_dense(a, nullptr).bytes;
    return static_cast<size_t>(4 * most_part_floats(kForward, a.type, a.pair, a.n, a.d_out, a.d_in, 1, 1)) + 256;
}

hipError_t launch_dense(const DenseArgs &a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    ProductArgs p{};
    p.a[0] = a.x;
    p.ld_a = a.ld_x;
    p.ld_b = a.ld_w;
    p.rows = a.n;
    p.cols = a.d_out;
    p.k = a.d_in;
    p.d_n = a.d_n;
    p.segs = p.short_segs = 1;
    p.products = 1;
    p.e.act = a.act;
    p.e.res = a.res;
    p.e.ld_res = a.ld_res;
    p.e.out[0] = a.out;
    p.e.ld_out = a.ld_out;
    p.e.ld_pre = a.ld_pre;
    for (int z = 0; z < 2; ++z) {
        p.b[z][0] = a.w[z];
        p.e.bias[z] = a.bias[z];
        p.e.pre[z] = a.pre[z];
    }
    return product(p, kForward, a.type, a.pair, a.ws, s);
}

hipError_t launch_dense_backward(const DenseArgs &a, hipStream_t s) {
    const int mats = a.pair ? 2 : 1;
    const bool bf = a.type == GNN_BF16, own = a.pair || a.act != GNN_ACT_NONE;      // dz is not dout itself
    const DenseSpace w = carve_dense(a, a.ws);
    const bool summed = a.dbias[0] || a.dbias[1];
    const int64_t size = bf ? 2 : 4;
    if (summed || (own && (a.dx || a.dw[0] || a.dw[1]))) {
        SlopeArgs p{};
        p.dout = a.dout;
        p.ld_dout = a.ld_dout;
        p.pre[0] = a.pre[0];
        p.pre[1] = a.pre[1];
        p.ld_pre = a.ld_pre;
        p.d_n = a.d_n;
        p.n = a.n;
        p.cols = a.d_out;
        p.act = a.act;
        p.store = own;
        p.planes_wide = w.wide;
        p.dz = w.dz;
        p.rest = w.rest;
        p.ld_dz = w.ld_dz;
        p.second = w.second;
        p.sums = summed ? reinterpret_cast<float *>(w.sums) : nullptr;
        p.ld_sums = w.ld_dz;
        hipError_t err = bf ? launch_slopes<bf16>(p, a.pair, s) : launch_slopes<float>(p, a.pair, s);
        if (err != hipSuccess) return err;
        if (summed) {
            err = launch_column_sums(p.sums, p.ld_sums, slope_parts(a.n, a.d_out, a.type), a.d_out, w.second, a.type,
                                     a.dbias[0], a.dbias[1], s);
            if (err != hipSuccess) return err;
        }
    }
    // Planes and projections of dz: index 2 plane + projection.
    const void *dz[4];
    for (int i = 0; i < 4; ++i)
        dz[i] = own ? (i < 2 ? w.dz : w.rest) + (i & 1) * w.second * size : static_cast<const char *>(a.dout);
    const int64_t ld_dz = own ? w.ld_dz : a.ld_dout;
    ProductArgs p{};
    p.d_n = a.d_n;
    p.e.act = GNN_ACT_NONE;
    if (a.dx && a.n > 0) {
        ProductArgs q = p;
        q.rows = a.n;
        q.cols = a.d_in;
        q.k = a.d_out;
        q.ld_a = ld_dz;
        q.ld_b = a.ld_w;
        q.segs = q.short_segs = mats;
        if (own && w.wide) q.segs = q.short_segs = 2 * mats;
        for (int i = 0; i < q.segs; ++i) {
            q.a[i] = a.pair ? dz[i] : dz[2 * i];
            q.b[0][i] = a.w[a.pair ? i & 1 : 0];
        }
        q.products = 1;
        q.e.out[0] = a.dx;
        q.e.ld_out = a.ld_dx;
        const hipError_t err = product(q, kGradX, a.type, false, w.part, s);
        if (err != hipSuccess) return err;
    }
    if (a.dw[0] || a.dw[1]) {
        ProductArgs q = p;
        q.rows = a.d_in;
        q.cols = a.d_out;
        q.k = a.n;
        q.ld_a = a.ld_x;
        q.ld_b = ld_dz;
        q.segs = 1;
        q.short_segs = own && bf ? 2 : 1;
        q.a[0] = q.a[1] = a.x;
        q.products = 0;
        q.e.ld_out = a.ld_dw;
        for (int z = 0; z < mats; ++z) {
            if (!a.dw[z]) continue;
            q.b[q.products][0] = dz[z];
            q.b[q.products][1] = dz[2 + z];
            q.e.out[q.products++] = a.dw[z];
        }
        const hipError_t err = product(q, kGradW, a.type, false, w.part, s);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace gnnmb
