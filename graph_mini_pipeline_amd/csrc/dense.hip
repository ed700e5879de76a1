// Dense layers on the matrix cores: y = act(x W + b) + r, the gated pair y = act(x Wg + bg) (x Wu + bu),
// and their gradients.
//
// Forward is one product with its epilogue (dense.hpp); a gated layer's two products share the tiles of x
// and meet in the epilogue's registers.  Backward, with z kept by the forward pass:
//   dz = dy act'(z)                 (k_slopes; gated: dg = dy u act'(g), du = dy act(g))
//   db = the sums of dz's columns   (partial sums by k_slopes, joined by the last workgroups of k_gradients)
//   dx = dz W^T, dW = x^T dz        (gated: dx = dg Wg^T + du Wu^T in one product over two segments)
// Without an activation dz is dy itself.
//
// Numbers.  Products are summed in fp32: bf16 on the 16-bit matrix instructions, fp32 on the fp32 ones.
// The dz of a bf16 layer is rounded to bf16 for its products, which leaves gradients 1.4 times as far from exact
// as their own rounding does (2.3e-3 for 1.7e-3 in the 2-norm), twice as far where few terms are summed; a sum of
// fewer than kShortSum terms takes dz in two planes, its bf16 and the bf16 of what that leaves (1.7e-3).  (In two planes
// everywhere, gradients of 16384 x 1024 x 4096 take 762 us for 309, gated 8192 x 2048 x 5632 1417 for 731.)  No
// atomic touches a sum: the parts of a split sum are added in their order.
//
// What it takes (us a call among others; in brackets the time at 5.4 TB/s, 1360 TFLOP/s in bf16 and 153 in fp32, which a
// copy of 512 MiB and the library's products of 8192 squares reach on the same card):
//   16384 x 4096 x 4096 bf16 with a residual 483 (404; the library's product alone 424), gated 16384 x 4096 x 10240 with
//   both sums kept 2316 (2021; the library's product of both weights alone 2077): the matrix units.
//   Gradients of 16384 x 1024 x 4096 bf16 with gelu 319 (202): dz 71, products 237, join 9; gated 8192 x 2048 x 5632
//   743 (556), of it dz 77.
//   One row, 4096 x 4096 bf16 13.5 (6.3): two launches, W at 3.4 TB/s.  Four rows, gated 4096 x 10240 36.0 (31.4).
//   333 x 1030 x 2571 fp32 with gelu and a residual 30.8 (11.5): a tile each for 246 compute units, loads by words;
//   gradients of 16384 x 256 x 128 fp32 43.2 (14.0) and gated 77 x 515 x 1371 fp32 27.6 (2.8): three launches of a few
//   dependent turns each.
// (Without matrix instructions, W read straight into registers by strips of columns over the whole summed length: one
// row of 4096 x 4096 13.5 us too, of 4096 x 10240 33 for 25, four rows 29 for 15; it was left.)
#include "dense.hpp"

namespace gnnmb {

namespace {

constexpr int kCus = 256;

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

constexpr int kColumnThreads = 1024;

__global__ __launch_bounds__(kColumnThreads) void k_column_sums(ColumnArgs p) {
    __shared__ float lds[kColumnThreads / 32 * 33];
    column_sums<kColumnThreads>(p, blockIdx.x, lds);
}

// ---- parts of a summed length, joined ------------------------------------------------------------------

// A workgroup takes 256 / L groups of four columns; L threads of each take every L-th part.
template <typename T, bool PAIR>
__device__ __forceinline__ void join_parts(const ProductArgs &p, int64_t rows, int lanes_log2, uint32_t block,
                                           vec<float, 4> *lds) {
    const uint32_t t = threadIdx.x, wide = 256u >> lanes_log2, lanes = 1u << lanes_log2;
    const uint32_t groups = static_cast<uint32_t>(p.ld_part >> 2), height = static_cast<uint32_t>(p.rows);
    const uint32_t e = block * wide + (t & (wide - 1)), lane = t >> (8 - lanes_log2);
    const uint32_t line = e / groups, z = line / height;
    const int64_t m = line - z * height, n = (e - line * groups) * 4;
    const bool there = z < (PAIR ? 1u : static_cast<uint32_t>(p.products)) && m < rows;
    const int64_t plane = static_cast<int64_t>(p.rows) * p.ld_part, products = PAIR ? 2 : p.products;
    vec<float, 4> v(0.f), u(0.f);
    if (there) {
        const float *from = p.part + (lane * products + z) * plane + m * p.ld_part + n;
        const int64_t step = lanes * products * plane;
#pragma unroll 4
        for (int s = lane; s < p.splits; s += lanes, from += step) {
            v += *reinterpret_cast<const vec<float, 4> *>(from);
            if (PAIR) u += *reinterpret_cast<const vec<float, 4> *>(from + plane);
        }
    }
    if (lanes > 1) {
        lds[t] = v;
        if (PAIR) lds[256 + t] = u;
        __syncthreads();
        if (lane == 0) {
            for (uint32_t i = 1; i < lanes; ++i) {
                v += lds[i * wide + t];
                if (PAIR) u += lds[256 + i * wide + t];
            }
        }
    }
    if (there && lane == 0)
        finish<T, 4, PAIR>(p.e, static_cast<int>(z), m, n, p.cols - n, v, u,
                           load_addends<T, 4, PAIR>(p.e, static_cast<int>(z), m, n, p.cols - n));
}

struct JoinArgs {
    ProductArgs p[2];
    int32_t lanes_log2[2];
    uint32_t blocks0;            // workgroups of p[0]
};

// FORWARD: p[0] alone, its rows counted by d_n.  Otherwise p[0] is of dW, p[1] of dx.
template <typename T, bool FORWARD, bool PAIR>
__global__ __launch_bounds__(256) void k_product_join(JoinArgs a) {
    __shared__ vec<float, 4> lds[PAIR ? 512 : 256];
    if (FORWARD || blockIdx.x < a.blocks0)
        join_parts<T, PAIR>(a.p[0], FORWARD ? load_count(a.p[0].d_n, a.p[0].rows) : a.p[0].rows, a.lanes_log2[0], blockIdx.x, lds);
    else
        join_parts<T, PAIR>(a.p[1], load_count(a.p[1].d_n, a.p[1].rows), a.lanes_log2[1], blockIdx.x - a.blocks0, lds);
}

// Threads a group of columns, and workgroups: eight threads for many parts where that fills the card.
uint32_t join_blocks(const ProductArgs &a, bool pair, int32_t *lanes_log2) {
    const int64_t groups = (pair ? 1 : a.products) * a.rows * (a.ld_part >> 2);
    *lanes_log2 = a.splits >= 8 && groups < 512 * kCus ? 3 : 0;
    const int64_t wide = 256 >> *lanes_log2;
    return static_cast<uint32_t>((groups + wide - 1) / wide);
}

// ---- planning ------------------------------------------------------------------------------------------

// The largest unit (16, 4 or 2 bytes) that all operands' lines are multiples of, as the way of their tiles
// into LDS.
int way_of(const ProductArgs &a, int form, bool pair, int size) {
    const int segs = a.segs > a.short_segs ? a.segs : a.short_segs;
    uint64_t bits = static_cast<uint64_t>((a.ld_a | a.ld_b) * size);
    for (int i = 0; i < segs; ++i) {
        bits |= reinterpret_cast<uintptr_t>(a.a[i]);
        for (int z = 0; z < (pair ? 2 : a.products); ++z) bits |= reinterpret_cast<uintptr_t>(a.b[z][i]);
    }
    if (form == kGradW) bits |= static_cast<uint64_t>(a.rows * size);
    if (form != kGradX) bits |= static_cast<uint64_t>(a.cols * size);
    return bits % 16 == 0 ? kByPiece : bits % 4 == 0 ? kByWord : kThrough;
}

// A product to be planned.
struct Shape {
    int form;
    int64_t rows, cols, k;
    int segs, products;
};

// What a workgroup takes, in us: its share of a compute unit that is full of such, for 128 bytes of the summed length
// (step) and besides, for the first loads and the epilogue (busy); and the same where it has the unit to itself (alone,
// fixed).  Measured on products of 1024 to 8192 rows and columns and on single rows.
struct TileCost {
    double step, busy, alone, fixed;
};
constexpr TileCost kCostBf16[4] = {{1.65, 8, 1.4, 8}, {0.62, 5, 0.62, 5}, {0.24, 1, 0.26, 2}, {0.24, 1.6, 0.27, 2}};
constexpr TileCost kCostF32[4] = {{0, 0, 0, 0}, {2.05, 5, 2.0, 4}, {0.56, 1.8, 0.58, 1.2}, {0.56, 1.8, 0.6, 1.2}};

// Parts of a sum are written and read again, at 3 TB/s, by a launch of its own (which behind the gradients' two
// others is waited for longer).
constexpr double kJoinLaunch = 3.0, kGradJoinLaunch = 4.0;
double join_us(int64_t parts, double elements) { return kJoinLaunch + static_cast<double>(parts) * elements * (8e-6 / 3.0); }

// The parts of a product take at most what 2048 tiles of 128 x 128 do, half of what the card's last cache holds: a
// workspace serves every smaller batch, so each large layer's has room for that much.  (Tiles of 256 alone could take
// more, up to 0.5 GB, for deep sums: 8782 x 16384 x 4096 bf16 1143 us by parts of 288 MB, 1193 without; of 200000 drawn
// shapes 95 forward plans lose over 3% by the time model, gradients none.)
constexpr int64_t kMostPartBytes = int64_t(128) << 20;

constexpr int kSplitChoices = 12;
constexpr int64_t kSplits[kSplitChoices] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

// What a product costs in so many parts.
struct Split {
    double groups, each;       // workgroups, steps of each
    double chain, work;        // us: of one workgroup, of all of them on one compute unit
    double join;
    bool sensible;
};

int64_t steps_of(const Shape &s, int type) {
    const int bk = type == GNN_BF16 ? 64 : 32;
    return (s.k + bk - 1) / bk * s.segs;
}

// Bytes of the parts for each row.
int64_t part_row_bytes(const Shape &s, bool pair, int64_t parts) { return 4 * parts * s.products * (pair ? 2 : 1) * round_up(s.cols, 4); }

// Up to how many rows so many parts are sensible.
int64_t split_rows(const Shape &s, int tile, bool pair, int64_t parts) {
    const int64_t tc = tile_cols(tile, pair), across = (s.cols + tc - 1) / tc * s.products * parts;
    const int64_t filled = 8 * kCus / across * tile_rows(tile), held = kMostPartBytes / part_row_bytes(s, pair, parts);
    return filled < held ? filled : held;
}

Split split_cost(const Shape &s, int type, int tile, bool pair, int64_t parts) {
    const TileCost &c = type == GNN_BF16 ? kCostBf16[tile] : kCostF32[tile];
    const int64_t tr = tile_rows(tile), tc = tile_cols(tile, pair);
    const int64_t tiles = ((s.rows + tr - 1) / tr) * ((s.cols + tc - 1) / tc) * s.products;
    const int64_t steps = steps_of(s, type);
    const double elements = static_cast<double>(s.rows) * s.cols * s.products * (pair ? 2 : 1);
    Split r;
    r.sensible = parts == 1 || (parts <= steps && s.rows <= split_rows(s, tile, pair, parts));
    r.groups = static_cast<double>(tiles * parts);
    r.each = static_cast<double>((steps + parts - 1) / parts);
    r.chain = r.each * c.alone + c.fixed;
    r.work = r.groups * (r.each * c.step + c.busy);
    r.join = parts > 1 ? join_us(parts, elements) : 0.0;
    return r;
}

// Bytes of the parts at most, of a product of up to s.rows rows; kGradW: of s.rows rows, and up to s.k summed ones.
int64_t most_part_bytes(const Shape &s, int type, int tile, bool pair) {
    int64_t most = 0;
    for (const int64_t parts : kSplits) {
        if (parts > steps_of(s, type)) break;
        int64_t rows = split_rows(s, tile, pair, parts);
        if (rows > s.rows) rows = s.rows;
        if (parts == 1 || (s.form == kGradW && rows < s.rows)) continue;
        const int64_t bytes = rows * part_row_bytes(s, pair, parts);
        if (bytes > most) most = bytes;
    }
    return most;
}

struct ForwardPlan {
    int tile;
    bool pair;         // one workgroup has both sums
    int64_t parts;
    bool joined;
};

constexpr int64_t kFewestRows = 64;       // up to which tiles of 32 rows are looked at

// Tiles of 64 and 32 take a gated pair as two products, whose sums are joined even where they are in one part.
bool is_apart(const DenseArgs &a, int tile) { return a.pair && tile > kTile128; }
Shape forward_shape(const DenseArgs &a, int tile) { return {kForward, a.n, a.d_out, a.d_in, 1, is_apart(a, tile) ? 2 : 1}; }

ForwardPlan plan_forward(const DenseArgs &a) {
    ForwardPlan best{};
    double least = 1e30;
    for (int tile = a.type == GNN_BF16 ? kTile256 : kTile128; tile <= kTile32; ++tile) {
        if (tile == kTile32 && a.n > kFewestRows) continue;
        const TileCost &c = a.type == GNN_BF16 ? kCostBf16[tile] : kCostF32[tile];
        const bool apart = is_apart(a, tile), pair = a.pair && !apart;
        const Shape shape = forward_shape(a, tile);
        if (apart && a.n * part_row_bytes(shape, false, 1) > kMostPartBytes) continue;
        for (const int64_t parts : kSplits) {
            const Split s = split_cost(shape, a.type, tile, pair, parts);
            if (!s.sensible) break;
            // the last round of workgroups may leave compute units idle
            const double rounds = static_cast<double>((static_cast<int64_t>(s.groups) + kCus - 1) / kCus);
            double us = rounds <= 1 ? s.chain : rounds * (s.each * c.step + c.busy);
            if (us < s.chain) us = s.chain;
            us += apart && parts == 1 ? join_us(1, 2.0 * static_cast<double>(a.n) * a.d_out) : s.join;
            if (us < least) {
                least = us;
                best = {tile, pair, parts, parts > 1 || apart};
            }
        }
    }
    return best;
}

// What the parts of a call of up to a.n rows take.
int64_t most_forward_bytes(DenseArgs a) {
    int64_t most = 0;
    for (int tile = a.type == GNN_BF16 ? kTile256 : kTile128; tile <= kTile32; ++tile) {
        if (tile == kTile32 && a.n > kFewestRows) a.n = kFewestRows;
        const bool apart = is_apart(a, tile);
        const Shape shape = forward_shape(a, tile);
        int64_t bytes = most_part_bytes(shape, a.type, tile, a.pair && !apart);
        if (apart) {
            const int64_t each = part_row_bytes(shape, false, 1), rows = kMostPartBytes / each;
            const int64_t whole = (a.n < rows ? a.n : rows) * each;
            if (whole > bytes) bytes = whole;
        }
        if (bytes > most) most = bytes;
    }
    return most;
}

struct GradientPlan {
    int tile;
    int64_t w_parts, x_parts;
};

// Both products' workgroups run in one launch: their parts are chosen together.
// dW of a few rows does without tiles, and takes what it writes.
GradientPlan plan_gradients(const Shape &w, const Shape &x, int type, bool few) {
    GradientPlan best{};
    double least = 1e30;
    const double written = static_cast<double>(w.rows) * w.cols * w.products * (type == GNN_BF16 ? 2 : 4);
    for (int tile = type == GNN_BF16 ? kTile256 : kTile128; tile <= kTile64; ++tile) {
        Split sx[kSplitChoices];
        for (int i = 0; i < kSplitChoices; ++i) sx[i] = split_cost(x, type, tile, false, kSplits[i]);
        for (const int64_t w_parts : kSplits) {
            Split sw = split_cost(w, type, tile, false, w_parts);
            if (few) {
                sw.sensible = w_parts == 1;
                sw.chain = 2.0;
                sw.work = written * (kCus * 1e-6 / 4.0);
            }
            if (!sw.sensible) break;
            for (int i = 0; i < kSplitChoices && sx[i].sensible; ++i) {
                const double chain = sw.chain > sx[i].chain ? sw.chain : sx[i].chain;
                const double shorter = sw.chain > sx[i].chain ? sx[i].chain : sw.chain;
                double us = (sw.work + sx[i].work) / kCus;
                if (sw.groups + sx[i].groups > kCus) us += 0.25 * shorter;      // of the last ones
                if (us < chain) us = chain;
                us += sw.join + sx[i].join;
                if (sw.join > 0 || sx[i].join > 0) us += kGradJoinLaunch - (sw.join > 0 && sx[i].join > 0 ? 2 : 1) * kJoinLaunch;
                if (us < least) {
                    least = us;
                    best = {tile, w_parts, kSplits[i]};
                }
            }
        }
    }
    return best;
}

// Only pieces fill the largest tile.
int filled_tile(int tile, int load) { return tile == kTile256 && load != kByPiece ? kTile128 : tile; }

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

// Each thread takes 16 bytes of a line; what it loads stays as it was loaded until its row's turn.  A line's last
// columns are taken by a piece that overlaps the one before: what both compute is the same, and counts in one's
// sums.  (SINGLE: lines shorter than a piece, element by element.)
template <typename T, bool PAIR, bool SINGLE>
__global__ __launch_bounds__(kSlopeWide * kSlopeHigh) void k_slopes(SlopeArgs p) {
    constexpr int V = SINGLE ? 1 : 16 / static_cast<int>(sizeof(T));
    constexpr bool kFast = sizeof(T) == 2;
    typedef vec<float, V> Wide;
    typedef vec<T, V> Raw;
    typedef typename loose<T, V>::type Loose;
    const int64_t n = load_count(p.d_n, p.n);
    const bool planes = kFast && (p.planes_wide || n < kShortSum);
    const int x = threadIdx.x % kSlopeWide, y = threadIdx.x / kSlopeWide;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kSlopeWide + x) * V;
    const int64_t c = at < p.cols - V ? at : p.cols - V;
    const bool there = at < p.cols;
    Wide sum0(0.f), sum1(0.f);
    const int64_t step = static_cast<int64_t>(gridDim.y) * kSlopeHigh;
    const auto load = [](const void *from, int64_t e) { return *reinterpret_cast<const Loose *>(static_cast<const T *>(from) + e); };
    const auto keep = [&](int64_t e, Wide v) {
        const Raw r = __builtin_convertvector(v, Raw);
        *reinterpret_cast<Loose *>(static_cast<T *>(p.dz) + e) = r;
        if (planes) {
            Wide rest = v - __builtin_convertvector(r, Wide);
            // An infinity leaves nothing: the difference would turn it into NaN.
#pragma unroll
            for (int i = 0; i < V; ++i) rest[i] = __builtin_fabsf(rest[i]) < __builtin_inff() ? rest[i] : 0.f;
            *reinterpret_cast<Loose *>(static_cast<T *>(p.rest) + e) = __builtin_convertvector(rest, Raw);
        }
    };
    if (there) {
        for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kSlopeHigh + y; m0 < n; m0 += step * kSlopeRows) {
            Raw d[kSlopeRows], a[kSlopeRows], b[kSlopeRows];
#pragma unroll
            for (int i = 0; i < kSlopeRows; ++i) {
                // past the end the first row again, which then counts for nothing
                const int64_t m = m0 + i * step < n ? m0 + i * step : m0;
                d[i] = load(p.dout, m * p.ld_dout + c);
                if (p.store) a[i] = load(p.pre[0], m * p.ld_pre + c);
                if (PAIR) b[i] = load(p.pre[1], m * p.ld_pre + c);
            }
#pragma unroll
            for (int i = 0; i < kSlopeRows; ++i) {
                const int64_t m = m0 + i * step;
                if (m >= n) break;
                const Wide dy = __builtin_convertvector(d[i], Wide);
                Wide g = dy;
                if (p.store) {
                    Wide z = __builtin_convertvector(a[i], Wide);
                    const Wide slope = activate_slope<kFast, V>(p.act, z);
                    g = PAIR ? dy * __builtin_convertvector(b[i], Wide) * slope : dy * slope;
                    keep(m * p.ld_dz + c, g);
                    if (PAIR) {
                        const Wide u = dy * z;
                        keep(m * p.ld_dz + p.second + c, u);
                        sum1 += u;
                    }
                }
                sum0 += g;
            }
        }
    }
    if (p.sums == nullptr) return;
    constexpr int kSums = (PAIR ? 2 : 1) * V;
    __shared__ float lds[kSlopeHigh][kSums][kSlopeWide + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        lds[y][i][x] = sum0[i];
        if (PAIR) lds[y][V + i][x] = sum1[i];
    }
    __syncthreads();
    for (int e = y; e < kSums; e += kSlopeHigh) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSlopeHigh; ++i) s += lds[i][e][x];
        if (there) p.sums[blockIdx.y * p.ld_sums + (e >= V ? p.second : 0) + c + e % V] = s;
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

// What the backward pass keeps in its workspace.  dz has whole 128-byte lines; of its second plane only what a
// short sum reads is there.
struct DenseSpace {
    char *dz, *rest, *sums, *w_part, *x_part;
    int64_t ld_dz, second;
    bool wide;               // two planes of every row: dx sums few terms
    bool few;                // dW by outer_tile
    Shape w, x;
    GradientPlan plan;
    size_t bytes;
};

// most: as large as any call of up to a.n rows needs it.
DenseSpace carve_dense(const DenseArgs &a, char *ws, bool most = false) {
    DenseSpace s{};
    const int mats = a.pair ? 2 : 1;
    const bool bf = a.type == GNN_BF16;
    const int64_t size = bf ? 2 : 4;
    s.second = round_up(a.d_out, 128 / size);
    s.ld_dz = s.second * mats;
    s.wide = bf && a.d_out * mats < kShortSum;
    s.w = {kGradW, a.d_in, a.d_out, a.n, 1, mats};
    s.x = {kGradX, a.n, a.d_in, a.d_out, s.wide ? 2 * mats : mats, 1};
    s.few = a.n > 0 && a.n <= kFewRows && a.d_out >= 16 / size;
    if (!most) s.plan = plan_gradients(s.w, s.x, a.type, s.few);
    const auto parts_of = [&](const Shape &shape, int64_t parts) {
        int64_t bytes = parts > 1 ? shape.rows * part_row_bytes(shape, false, parts) : 0;
        for (int tile = bf ? kTile256 : kTile128; most && tile <= kTile64; ++tile) {
            const int64_t by_tile = most_part_bytes(shape, a.type, tile, false);
            if (by_tile > bytes) bytes = by_tile;
        }
        return bytes;
    };
    size_t at = 0;
    const auto take = [&](char **p, int64_t bytes) {
        *p = ws + at;
        at += static_cast<size_t>(round_up(bytes < 1 ? 1 : bytes, 256));
    };
    take(&s.dz, a.n * s.ld_dz * size);
    take(&s.rest, !bf ? 0 : (s.wide || a.n < kShortSum ? a.n : kShortSum) * s.ld_dz * size);
    take(&s.sums, static_cast<int64_t>(slope_parts(a.n, a.d_out, a.type)) * s.ld_dz * 4);
    take(&s.w_part, parts_of(s.w, s.plan.w_parts));
    take(&s.x_part, parts_of(s.x, s.plan.x_parts));
    s.bytes = at;
    return s;
}

template <typename T, bool PAIR>
hipError_t launch_slopes(const SlopeArgs &a, hipStream_t s) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const bool single = a.cols < V;
    const int64_t wide = kSlopeWide * (single ? 1 : V);
    const dim3 grid(static_cast<unsigned>((a.cols + wide - 1) / wide),
                    slope_parts(a.n, a.cols, sizeof(T) == 2 ? GNN_BF16 : GNN_F32));
    if (single)
        k_slopes<T, PAIR, true><<<grid, kSlopeWide * kSlopeHigh, 0, s>>>(a);
    else
        k_slopes<T, PAIR, false><<<grid, kSlopeWide * kSlopeHigh, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_column_sums(const float *sums, int64_t ld, int parts, int64_t cols, int64_t second, int type, void *out0,
                              void *out1, hipStream_t s) {
    const ColumnArgs c{sums, ld, parts, cols, second, type, {out0, out1}, static_cast<uint32_t>((cols + 31) / 32)};
    k_column_sums<<<2 * c.blocks, kColumnThreads, 0, s>>>(c);
    return hipGetLastError();
}

size_t dense_bytes(const DenseArgs &a, bool backward) {
    return backward ? carve_dense(a, nullptr, true).bytes : 256 + static_cast<size_t>(most_forward_bytes(a));
}

hipError_t launch_dense(const DenseArgs &a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    const bool bf = a.type == GNN_BF16;
    const ForwardPlan plan = plan_forward(a);
    JoinArgs j{};
    ProductArgs &p = j.p[0];
    p.a[0] = a.x;
    p.ld_a = a.ld_x;
    p.ld_b = a.ld_w;
    p.rows = a.n;
    p.cols = a.d_out;
    p.k = a.d_in;
    p.d_n = a.d_n;
    p.segs = p.short_segs = 1;
    p.products = 1;
    p.splits = static_cast<int32_t>(plan.parts);
    p.part = plan.joined ? reinterpret_cast<float *>(a.ws) : nullptr;
    p.ld_part = round_up(a.d_out, 4);
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
    const int load = way_of(p, kForward, a.pair, bf ? 2 : 4);
    ProductArgs q = p;
    if (a.pair && !plan.pair) q.products = 2;
    const int tile = filled_tile(plan.tile, load);
    const hipError_t err = bf ? launch_product_bf16(q, tile, plan.pair, load, s) : launch_product_f32(q, tile, plan.pair, load, s);
    if (err != hipSuccess || !plan.joined) return err;
    const uint32_t blocks = join_blocks(p, a.pair, &j.lanes_log2[0]);
    if (bf && a.pair)
        k_product_join<bf16, true, true><<<blocks, 256, 0, s>>>(j);
    else if (bf)
        k_product_join<bf16, true, false><<<blocks, 256, 0, s>>>(j);
    else if (a.pair)
        k_product_join<float, true, true><<<blocks, 256, 0, s>>>(j);
    else
        k_product_join<float, true, false><<<blocks, 256, 0, s>>>(j);
    return hipGetLastError();
}

hipError_t launch_dense_backward(const DenseArgs &a, hipStream_t s) {
    const int mats = a.pair ? 2 : 1;
    const bool bf = a.type == GNN_BF16, own = a.pair || a.act != GNN_ACT_NONE;      // dz is not dout itself
    const DenseSpace w = carve_dense(a, a.ws);
    const bool summed = a.dbias[0] || a.dbias[1], weights = a.dw[0] || a.dw[1], inputs = a.dx && a.n > 0;
    const int64_t size = bf ? 2 : 4;
    if (!summed && !weights && !inputs) return hipSuccess;
    ColumnArgs c{};
    if (summed || own) {
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
        const hipError_t err = a.pair ? (bf ? launch_slopes<bf16, true>(p, s) : launch_slopes<float, true>(p, s))
                                      : (bf ? launch_slopes<bf16, false>(p, s) : launch_slopes<float, false>(p, s));
        if (err != hipSuccess) return err;
        if (summed)
            c = ColumnArgs{p.sums, p.ld_sums, slope_parts(a.n, a.d_out, a.type), a.d_out, w.second, a.type,
                           {a.dbias[0], a.dbias[1]}, static_cast<uint32_t>((a.d_out + 31) / 32)};
    }
    // Planes and projections of dz: index 2 plane + projection.
    const void *dz[4];
    for (int i = 0; i < 4; ++i)
        dz[i] = own ? (i < 2 ? w.dz : w.rest) + (i & 1) * w.second * size : static_cast<const char *>(a.dout);
    const int64_t ld_dz = own ? w.ld_dz : a.ld_dout;
    JoinArgs j{};
    ProductArgs &pw = j.p[0], &px = j.p[1];
    const auto sized = [&](ProductArgs &q, const Shape &shape, int64_t parts, char *part) {
        q.rows = shape.rows;
        q.cols = shape.cols;
        q.k = shape.k;
        q.d_n = a.d_n;
        q.splits = static_cast<int32_t>(parts);
        q.part = parts > 1 ? reinterpret_cast<float *>(part) : nullptr;
        q.ld_part = round_up(q.cols, 4);
        q.e.act = GNN_ACT_NONE;
    };
    // Segments: those of the second plane, where there is one, before the first's.
    sized(pw, w.w, w.plan.w_parts, w.w_part);
    pw.ld_a = a.ld_x;
    pw.ld_b = ld_dz;
    pw.segs = 1;
    pw.rest = own && bf ? 1 : 0;
    pw.short_segs = 1 + pw.rest;
    pw.a[0] = pw.a[1] = a.x;
    pw.e.ld_out = a.ld_dw;
    pw.few = !w.few ? 0 : bf ? kOuterWide<bf16> : kOuterWide<float>;
    for (int z = 0; z < mats; ++z) {
        if (!a.dw[z]) continue;
        pw.b[pw.products][0] = dz[2 * pw.rest + z];
        pw.b[pw.products][1] = dz[z];
        pw.e.out[pw.products++] = a.dw[z];
    }
    sized(px, w.x, w.plan.x_parts, w.x_part);
    px.ld_a = ld_dz;
    px.ld_b = a.ld_w;
    px.rest = own && w.wide ? mats : 0;
    px.segs = px.short_segs = px.rest + mats;
    for (int i = 0; i < px.segs; ++i) {
        px.a[i] = dz[(i < px.rest ? 2 : 0) + i % mats];
        px.b[0][i] = a.w[i % mats];
    }
    px.products = inputs ? 1 : 0;
    px.e.out[0] = a.dx;
    px.e.ld_out = a.ld_dx;
    const int way_w = weights && !w.few ? way_of(pw, kGradW, false, size) : kByPiece;
    const int way_x = inputs ? way_of(px, kGradX, false, size) : kByPiece;
    const int load = way_w > way_x ? way_w : way_x, tile = filled_tile(w.plan.tile, load);
    hipError_t err = bf ? launch_gradients_bf16(pw, px, c, tile, load, s) : launch_gradients_f32(pw, px, c, tile, load, s);
    if (err != hipSuccess) return err;
    j.blocks0 = pw.part && weights ? join_blocks(pw, false, &j.lanes_log2[0]) : 0;
    const uint32_t blocks = j.blocks0 + (px.part && inputs ? join_blocks(px, false, &j.lanes_log2[1]) : 0);
    if (blocks == 0) return hipSuccess;
    if (bf)
        k_product_join<bf16, false, false><<<blocks, 256, 0, s>>>(j);
    else
        k_product_join<float, false, false><<<blocks, 256, 0, s>>>(j);
    return hipGetLastError();
}

}  // namespace gnnmb
