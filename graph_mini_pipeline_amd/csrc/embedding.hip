// Embedding lookup with scaling, and its gradient by sorted ids.
//
// Lookup: out[i, :] = scale * table[ids[i], :], one rounding to the output's type.  Memory-bound: a
// thread holds kLookUnroll independent 16-byte row pieces in flight.  1081344 rows of 100 fp32 to bf16:
// 135 us, 4.8 TB/s of rows and results, what a large copy reaches; 16384 x 768 bf16 8 us on the device.
//
// Gradient: G[t, :] = scale * sum over the positions i with ids[i] = t of dout[i, :], for a dense
// table or for the distinct ids only.  The (id, position) pairs are sorted by id, stably, so that
// each id's positions follow each other in ascending order; then
//   - the sorted list is cut into chunks of equal length, whatever the ids' frequencies, so a word
//     that holds a tenth of all positions costs no more than any other tenth: a lane group walks
//     one chunk, keeps one fp32 sum per column in registers, and stores it whenever the id changes.
//     A run that lies within the chunk is final; the chunk's first and last run may go on beyond
//     it, and leave a partial sum per chunk in the workspace;
//   - those are joined in chunk order: a run of two chunks by a lane group, a longer one, which the
//     first pass lists, by a workgroup.
// No atomic touches a sum, so results do not depend on timing.
//
// What bounds it: the reading of dout, in rows that lie apart.  131072 x 1024 bf16 over 50257 rows: sums 107
// us of 146 (4.3 TB/s of dout and the fp32 table), two digits of the sort 31, joining 10.  901120 x 100 fp32
// over 400000 nodes: sums 154 of 263 (rows of 400 bytes fetch 512), three digits 69, ids 12, joining 22.
// (Finishing a run of two chunks by the group that began it saves partial sums but makes the chunks'
// walks uneven: 139 + 10 us for 107 + 17 at the first shape, and was left.)
#include "learn.hpp"

namespace gnnmb {

namespace {

constexpr int kLookThreads = 256;
constexpr int kLookUnroll = 4;

template <typename TI, typename TO, int VE>
__global__ __launch_bounds__(kLookThreads) void k_embedding_lookup(LookupArgs a) {
    const int64_t n = load_count(a.d_n, a.n);
    const int64_t base = (a.first_block + blockIdx.x) * (kLookThreads * kLookUnroll);
    const int64_t row0 = base / a.cpr;
    if (row0 >= n) return;
    const uint32_t rem = static_cast<uint32_t>(base - row0 * a.cpr);
    const TI *table = static_cast<const TI *>(a.table);
    typename loose<TI, VE>::type v[kLookUnroll];
    int64_t row[kLookUnroll];
    int64_t col[kLookUnroll];
    bool live[kLookUnroll];
    // Every load is made, of a row that exists, so that none waits for a branch.
#pragma unroll
    for (int u = 0; u < kLookUnroll; ++u) {
        const uint32_t off = rem + u * kLookThreads + threadIdx.x;
        const uint32_t q = fast_div(off, a.by_cpr);
        row[u] = row0 + q;
        // the last piece of a row ends at its end: it overlaps the one before where VE does not
        // divide d, and both store the same values there
        col[u] = static_cast<int64_t>(off - q * a.cpr) * VE;
        if (col[u] > a.d - VE) col[u] = a.d - VE;
        const int32_t id = a.ids[row[u] < n ? row[u] : n - 1];
        const bool good = id >= 0 && id < a.num_rows;
        const bool pad = id >= 0 && id == a.pad_id;      // (which may lie outside the table)
        live[u] = good && !pad;
        if (!good && !pad && row[u] < n) set_status(a.status, GNN_ERR_OUT_OF_RANGE);
        v[u] = *reinterpret_cast<const typename loose<TI, VE>::type *>(
            table + static_cast<int64_t>(good ? id : 0) * a.ld + col[u]);
    }
    TO *out = static_cast<TO *>(a.out);
#pragma unroll
    for (int u = 0; u < kLookUnroll; ++u)
        if (row[u] < n) {
            const vec<float, VE> x = __builtin_convertvector(v[u], vec<float, VE>) * a.scale;
            store_f32<TO, VE>(out + row[u] * a.ld_out + col[u], live[u] ? x : vec<float, VE>(0.f));
        }
}

template <typename TI, typename TO, int VE>
hipError_t run_lookup(LookupArgs a, hipStream_t s) {
    a.cpr = static_cast<uint32_t>((a.d + VE - 1) / VE);
    a.by_cpr = make_fastdiv(a.cpr);
    const int64_t per = kLookThreads * kLookUnroll;
    return launch_pieces((a.n * a.cpr + per - 1) / per, kLookThreads, [&](int64_t first, unsigned blocks) {
        a.first_block = first;
        hipLaunchKernelGGL((k_embedding_lookup<TI, TO, VE>), dim3(blocks), dim3(kLookThreads), 0, s, a);
    });
}

template <typename TI, typename TO>
hipError_t pick_lookup(const LookupArgs &a, hipStream_t s) {
    // 16 bytes of the narrower type, unless rows end in a half-filled piece of 8
    constexpr bool wide = sizeof(TI) == 2 || sizeof(TO) == 2;
    if (wide && a.d >= 8 && (a.d % 8 == 0 || a.d % 8 > 4)) return run_lookup<TI, TO, 8>(a, s);
    if (a.d >= 4) return run_lookup<TI, TO, 4>(a, s);
    return run_lookup<TI, TO, 1>(a, s);
}

// ---- the sort -----------------------------------------------------------------------------------
//
// Least-significant-digit radix sort of (key, position) by digits of at most 8 bits, stable.  A
// workgroup takes a tile of keys, 8 per thread; a wavefront's keys lie next to each other, 64 a
// round, so the order (wavefront, round, lane) is the order of the positions.  Lanes with the same
// digit find each other by one ballot per bit of the digit.  Up to 8192 keys (of the distinct ids: a dense
// table of so few positions goes by buckets) are sorted by one
// workgroup of 16 wavefronts in LDS in one launch.  Beyond that, each digit takes two launches over
// tiles of 4096 keys: digit counts of every tile, then the placement, where every tile sums the
// counts of the tiles before it (beyond kSumTiles tiles a third launch does that once for all).
constexpr int kSortRounds = 8;
constexpr int kOneThreads = 1024;                       // the one-workgroup sort
constexpr int kOneTile = kOneThreads * kSortRounds;
constexpr int kSortThreads = 512;                       // the tiled sort
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortTile = kSortThreads * kSortRounds;
constexpr int kSortBits = 8;
constexpr int kDigits = 1 << kSortBits;
constexpr int kSumTiles = 256;
constexpr int64_t kChunkMin = 8;      // shortest chunk of the sums

struct SortArgs {
    const int32_t *ids;
    const int64_t *d_n;
    int64_t n;
    int32_t pad_id;
    uint32_t num_rows;      // also the key of positions without a gradient row: they sort last
    int32_t *status;
    const uint32_t *key_in, *pos_in;   // NULL: the first digit, read from ids
    uint32_t *key_out, *pos_out;
    uint32_t *hist;         // [tiles, kDigits], then (scanned) the digits' totals
    int32_t tiles;
    int32_t scanned;
    int32_t shift, bits;
    // work of other parts of the gradient that rides along
    uint8_t *touched;       // [num_rows] 1: some id names the row; cleared by the first count, marked
    int64_t touched_words;  // by the first placement; NULL: none
    uint32_t *long_runs;    // their number is cleared by the first count
    // run heads (the rows form)
    int32_t *uniq;
    int64_t *d_n_uniq;
    int64_t row_cap;
    uint32_t *chunk_rank;
    int32_t chunk;
    int32_t passes;
};

// The key of position i, which holds id.
__device__ __forceinline__ uint32_t make_key(const SortArgs &a, int64_t i, int64_t n_act, int32_t id) {
    if (i >= n_act || (id >= 0 && id == a.pad_id)) return a.num_rows;
    if (id < 0 || static_cast<uint32_t>(id) >= a.num_rows) {
        set_status(a.status, GNN_ERR_OUT_OF_RANGE);
        return a.num_rows;
    }
    return static_cast<uint32_t>(id);
}

// Clears the marks and the number of long runs; the grid's threads share the work.
__device__ __forceinline__ void clear_marks(const SortArgs &a) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (t == 0) *a.long_runs = 0;
    if (a.touched == nullptr) return;
    uint32_t *w = reinterpret_cast<uint32_t *>(a.touched);
    for (int64_t i = t; i < a.touched_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x) w[i] = 0;
}

// Ranks each round's keys among the wavefront's earlier keys of the same digit; cnt (this
// wavefront's digit counts, zero before) receives the counts.
template <int ROUNDS>
__device__ __forceinline__ void rank_rounds(const uint32_t (&key)[ROUNDS], int rounds, int shift,
                                            int bits, uint32_t *cnt, uint32_t (&rank)[ROUNDS]) {
    const uint64_t below = (1ull << lane_id()) - 1ull;
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        if (j >= rounds) break;
        const uint32_t dg = (key[j] >> shift) & ((1u << bits) - 1u);
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((dg >> b) & 1u);
            same &= ((dg >> b) & 1u) ? m : ~m;
        }
        const uint32_t before = cnt[dg];
        rank[j] = before + __popcll(same & below);
        wave_lds_sync();
        if ((same & below) == 0) cnt[dg] = before + __popcll(same);
        wave_lds_sync();
    }
}

// Exclusive scan of 256 values, one per thread of the first four wavefronts; every thread of the
// workgroup calls it (the others' v is ignored).
__device__ __forceinline__ uint32_t scan_digits(uint32_t v, uint32_t *s4) {
    const int w = threadIdx.x >> 6;
    const uint32_t inc = wave_inclusive_scan(v);
    if (w < 4 && lane_id() == 63) s4[w] = inc;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < 3; ++i)
        if (i < w) before += s4[i];
    __syncthreads();
    return before + inc - v;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs a) {
    __shared__ uint32_t h[kDigits];
    const int t = threadIdx.x;
    if (t < kDigits) h[t] = 0;
    if (a.key_in == nullptr) clear_marks(a);
    const int64_t n_act = load_count(a.d_n, a.n);
    const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * kSortTile;
    const int32_t *in = a.key_in ? reinterpret_cast<const int32_t *>(a.key_in) : a.ids;
    int32_t x[kSortRounds];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const int64_t i = tile0 + j * kSortThreads + t;
        x[j] = in[i < a.n ? i : a.n - 1];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const int64_t i = tile0 + j * kSortThreads + t;
        if (i >= a.n) continue;
        const uint32_t key = a.key_in ? static_cast<uint32_t>(x[j]) : make_key(a, i, n_act, x[j]);
        atomicAdd(&h[(key >> a.shift) & ((1u << a.bits) - 1u)], 1u);
    }
    __syncthreads();
    if (t < kDigits) a.hist[static_cast<int64_t>(blockIdx.x) * kDigits + t] = h[t];
}

// One workgroup per digit: exclusive prefix over the tiles, in place; the total at [tiles].
__global__ __launch_bounds__(256) void k_sort_scan(SortArgs a) {
    __shared__ uint32_t sm[4];
    const int dg = blockIdx.x;
    uint32_t carry = 0;
    for (int64_t t0 = 0; t0 < a.tiles; t0 += 256) {
        const int64_t t = t0 + threadIdx.x;
        const uint32_t v = t < a.tiles ? a.hist[t * kDigits + dg] : 0u;
        uint32_t total;
        const uint32_t ex = block_exclusive_scan<uint32_t, 256>(v, &total, sm);
        if (t < a.tiles) a.hist[t * kDigits + dg] = carry + ex;
        carry += total;
    }
    if (threadIdx.x == 0) a.hist[static_cast<int64_t>(a.tiles) * kDigits + dg] = carry;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs a) {
    __shared__ uint32_t cnt[kSortWaves][kDigits];
    __shared__ uint32_t sums[2][kSortThreads / kDigits][kDigits];
    __shared__ uint32_t base[kDigits], local[kDigits];
    __shared__ uint32_t skey[kSortTile], spos[kSortTile];
    __shared__ uint32_t s4[4];
    const int t = threadIdx.x, w = t >> 6;
    for (int i = t; i < kSortWaves * kDigits; i += kSortThreads) (&cnt[0][0])[i] = 0;
    const int64_t n_act = load_count(a.d_n, a.n);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTile + w * (64 * kSortRounds) +
                       lane_id();
    uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
    const bool given = a.key_in != nullptr;
    const int32_t *in = given ? reinterpret_cast<const int32_t *>(a.key_in) : a.ids;
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const int64_t i = i0 + j * 64 < a.n ? i0 + j * 64 : a.n - 1;
        key[j] = static_cast<uint32_t>(in[i]);
        pos[j] = given ? a.pos_in[i] : static_cast<uint32_t>(i);
    }
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const int64_t i = i0 + j * 64;
        if (i >= a.n) {
            key[j] = 0xffffffffu;        // beyond the end: ranked after every key of the last tile
        } else if (!given) {
            key[j] = make_key(a, i, n_act, static_cast<int32_t>(key[j]));
            if (a.touched && key[j] < a.num_rows) a.touched[key[j]] = 1;
        }
    }
    // counts of the tiles before this one and of all tiles, kSortThreads / kDigits threads per digit
    const int dg = t & (kDigits - 1), part = t / kDigits;
    uint32_t before = 0, total = 0;
    if (a.scanned) {
        if (part == 0) {
            before = a.hist[static_cast<int64_t>(blockIdx.x) * kDigits + dg];
            total = a.hist[static_cast<int64_t>(a.tiles) * kDigits + dg];
        }
    } else {
#pragma unroll 8
        for (int k = part; k < a.tiles; k += kSortThreads / kDigits) {
            const uint32_t c = a.hist[k * kDigits + dg];
            total += c;
            if (k < static_cast<int>(blockIdx.x)) before += c;
        }
    }
    sums[0][part][dg] = before;
    sums[1][part][dg] = total;
    __syncthreads();
    rank_rounds<kSortRounds>(key, kSortRounds, a.shift, a.bits, cnt[w], rank);
    __syncthreads();
    before = total = 0;
    uint32_t run = 0;
    if (t < kDigits) {
        for (int q = 0; q < kSortThreads / kDigits; ++q) {
            before += sums[0][q][t];
            total += sums[1][q][t];
        }
        for (int q = 0; q < kSortWaves; ++q) {
            const uint32_t c = cnt[q][t];
            cnt[q][t] = run;
            run += c;
        }
    }
    const uint32_t ex = scan_digits(total, s4);
    const uint32_t in_tile = scan_digits(run, s4);
    if (t < kDigits) {
        base[t] = ex + before - in_tile;      // from a place in the sorted tile to the place in the list
        local[t] = in_tile;
    }
    __syncthreads();
    // The tile is put in order in LDS first, so that a digit's keys leave it side by side: as single
    // words they would each cost the memory a whole line (901120 positions: 21 us a digit, this
    // way 18).
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const uint32_t g = (key[j] >> a.shift) & ((1u << a.bits) - 1u);
        const uint32_t to = local[g] + cnt[w][g] + rank[j];
        skey[to] = key[j];
        spos[to] = pos[j];
    }
    __syncthreads();
    const int64_t left = a.n - static_cast<int64_t>(blockIdx.x) * kSortTile;     // keys of this tile
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        const int i = j * kSortThreads + t;
        const uint32_t k = skey[i];
        // (past the end: the tile's last keys, which are no positions')
        if (i >= left) continue;
        const uint32_t to = base[(k >> a.shift) & ((1u << a.bits) - 1u)] + i;
        a.key_out[to] = k;
        a.pos_out[to] = spos[i];
    }
}

__device__ __forceinline__ bool is_head(uint32_t key, uint32_t prev, bool first, uint32_t rows) {
    return key < rows && (first || key != prev);
}

// The one-workgroup sort: n <= ROUNDS * THREADS positions, sorted, in key and pos.
template <int ROUNDS, int THREADS>
struct OneSort {
    static constexpr int kWaves = THREADS / 64;
    uint32_t key[ROUNDS * THREADS];
    uint16_t pos[ROUNDS * THREADS];
    uint32_t cnt[kWaves][kDigits];
    uint32_t base[kDigits];
    uint32_t s4[4];
};

// The thread's keys, in the order that the sort takes them.
template <int ROUNDS, int THREADS>
__device__ __forceinline__ void load_keys(const SortArgs &a, uint32_t (&key)[ROUNDS]) {
    const int n = static_cast<int>(a.n);
    const int64_t n_act = load_count(a.d_n, a.n);
    const int rounds = (n + THREADS - 1) / THREADS;
    const int i0 = (static_cast<int>(threadIdx.x) >> 6) * 64 * rounds + lane_id();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j)
        if (j < rounds) key[j] = static_cast<uint32_t>(a.ids[i0 + j * 64 < n ? i0 + j * 64 : n - 1]);
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        if (j >= rounds) continue;
        const int i = i0 + j * 64;
        // slots beyond n: after every position of the same key
        key[j] = i < n ? make_key(a, i, n_act, static_cast<int32_t>(key[j])) : a.num_rows;
    }
}

// The thread's positions, of the keys that load_keys() gives it.
template <int ROUNDS, int THREADS>
__device__ __forceinline__ void own_positions(int64_t n, uint32_t (&pos)[ROUNDS]) {
    const int rounds = (static_cast<int>(n) + THREADS - 1) / THREADS;
    const int i0 = (static_cast<int>(threadIdx.x) >> 6) * 64 * rounds + lane_id();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) pos[j] = static_cast<uint32_t>(i0 + j * 64);
}

// Every thread of the workgroup calls it, with its keys and their positions.
template <int ROUNDS, int THREADS>
__device__ __forceinline__ void sort_one(int n, int passes, int bits, OneSort<ROUNDS, THREADS> &m,
                                         uint32_t (&key)[ROUNDS], uint32_t (&pos)[ROUNDS]) {
    constexpr int kWaves = THREADS / 64;
    const int t = threadIdx.x, w = t >> 6;
    const int rounds = (n + THREADS - 1) / THREADS;
    const int i0 = w * 64 * rounds + lane_id();
    uint32_t rank[ROUNDS];
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        for (int i = t; i < kWaves * kDigits; i += THREADS) (&m.cnt[0][0])[i] = 0;
        __syncthreads();
        rank_rounds<ROUNDS>(key, rounds, shift, bits, m.cnt[w], rank);
        __syncthreads();
        uint32_t total = 0;
        if (t < kDigits) {
            uint32_t c[kWaves];
#pragma unroll
            for (int q = 0; q < kWaves; ++q) c[q] = m.cnt[q][t];
#pragma unroll
            for (int q = 0; q < kWaves; ++q) {
                m.cnt[q][t] = total;
                total += c[q];
            }
        }
        const uint32_t ex = scan_digits(total, m.s4);
        if (t < kDigits) m.base[t] = ex;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
            if (j >= rounds) continue;
            const uint32_t g = (key[j] >> shift) & ((1u << bits) - 1u);
            const uint32_t to = m.base[g] + m.cnt[w][g] + rank[j];
            m.key[to] = key[j];
            m.pos[to] = static_cast<uint16_t>(pos[j]);
        }
        __syncthreads();
        if (p + 1 == passes) break;
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
            if (j >= rounds) continue;
            key[j] = m.key[i0 + j * 64];
            pos[j] = m.pos[i0 + j * 64];
        }
    }
}

__global__ __launch_bounds__(kOneThreads) void k_sort_one(SortArgs a) {
    __shared__ OneSort<kSortRounds, kOneThreads> m;
    __shared__ uint32_t sw[kOneThreads / 64];
    const int t = threadIdx.x;
    const int n = static_cast<int>(a.n);
    uint32_t key[kSortRounds];
    load_keys<kSortRounds, kOneThreads>(a, key);
    if (t == 0) *a.long_runs = 0;
    uint32_t pos[kSortRounds];
    own_positions<kSortRounds, kOneThreads>(a.n, pos);
    sort_one(n, a.passes, a.bits, m, key, pos);
    for (int i = t; i < n; i += kOneThreads) {
        a.key_out[i] = m.key[i];
        a.pos_out[i] = m.pos[i];
    }
    uint32_t carry = 0;
    for (int r0 = 0; r0 < n; r0 += kOneThreads) {
        const int i = r0 + t;
        const uint32_t k = i < n ? m.key[i] : a.num_rows;
        const uint32_t head = is_head(k, i > 0 ? m.key[i < n ? i - 1 : 0] : 0u, i == 0, a.num_rows);
        uint32_t total;
        const uint32_t at = carry + block_exclusive_scan<uint32_t, kOneThreads>(head, &total, sw);
        if (head && at < a.row_cap) a.uniq[at] = static_cast<int32_t>(k);
        if (i < n && i % a.chunk == 0) a.chunk_rank[i / a.chunk] = at + head - 1u;
        carry += total;
    }
    if (t == 0) {
        *a.d_n_uniq = carry;
        if (carry > a.row_cap) set_status(a.status, GNN_ERR_CAPACITY);
    }
}

// The rows form beyond one tile: run heads of every tile, then the distinct ids.
struct HeadArgs {
    const uint32_t *key;
    int64_t n;
    uint32_t num_rows;
    uint32_t *heads;        // [tiles]
    int32_t tiles;
    int32_t *uniq;
    int64_t *d_n_uniq;
    int64_t row_cap;
    uint32_t *chunk_rank;
    int32_t chunk;
    int32_t *status;
};

__device__ __forceinline__ uint32_t tile_heads(const HeadArgs &a, int64_t i0, uint32_t &flags) {
    flags = 0;
    uint32_t prev = i0 > 0 && i0 < a.n ? a.key[i0 - 1] : 0u;
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        if (i0 + j >= a.n) break;
        const uint32_t k = a.key[i0 + j];
        if (is_head(k, prev, i0 + j == 0, a.num_rows)) flags |= 1u << j;
        prev = k;
    }
    return __popc(flags);
}

__global__ __launch_bounds__(kSortThreads) void k_count_heads(HeadArgs a) {
    __shared__ uint32_t sm[kSortWaves];
    uint32_t flags, total;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTile + threadIdx.x * kSortRounds;
    const uint32_t c = tile_heads(a, i0, flags);
    block_exclusive_scan<uint32_t, kSortThreads>(c, &total, sm);
    if (threadIdx.x == 0) a.heads[blockIdx.x] = total;
}

__global__ __launch_bounds__(kSortThreads) void k_emit_heads(HeadArgs a) {
    __shared__ uint32_t sm[kSortWaves];
    uint32_t mine = 0, before, flags, total;
    for (int k = threadIdx.x; k < static_cast<int>(blockIdx.x); k += kSortThreads) mine += a.heads[k];
    block_exclusive_scan<uint32_t, kSortThreads>(mine, &before, sm);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTile + threadIdx.x * kSortRounds;
    const uint32_t c = tile_heads(a, i0, flags);
    uint32_t at = before + block_exclusive_scan<uint32_t, kSortThreads>(c, &total, sm);
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
        if (i0 + j >= a.n) break;
        const bool head = (flags >> j) & 1u;
        if (head && at < a.row_cap) a.uniq[at] = static_cast<int32_t>(a.key[i0 + j]);
        at += head;
        if ((i0 + j) % a.chunk == 0) a.chunk_rank[(i0 + j) / a.chunk] = at - 1u;
    }
    if (static_cast<int>(blockIdx.x) == a.tiles - 1 && threadIdx.x == 0) {
        *a.d_n_uniq = static_cast<int64_t>(before) + total;
        if (static_cast<int64_t>(before) + total > a.row_cap) set_status(a.status, GNN_ERR_CAPACITY);
    }
}

// ---- the sums -----------------------------------------------------------------------------------

constexpr int kSumThreads = 256;
constexpr int kSumUnroll = 8;     // rows of dout in flight per lane
constexpr int kJoinRuns = 512;    // workgroups per slab that share the listed runs

struct SumArgs {
    const uint32_t *key, *pos;
    int64_t n;
    uint32_t num_rows;
    const void *dout;
    int64_t ld_dout, d;
    float scale;
    void *out;
    int64_t ld_out;
    int32_t accumulate;
    const uint32_t *chunk_rank;    // rows form
    int64_t row_cap;
    float *part;                   // [2 * chunks, d] sums of a chunk's first run (even) where it
                                   // began earlier, and of its last run (odd) where it goes on
    int32_t chunk;
    int64_t chunks;
    int32_t lanes;                 // lanes per chunk, a power of two
    int32_t slabs;                 // groups of lanes side by side along a row
    const uint8_t *touched;        // dense, written: rows without a mark are zeroed
    uint32_t *long_runs;           // number of listed runs, then their first chunks
    int64_t sum_blocks;            // blocks beyond these zero rows
};

// The columns of one lane: VE from `at`, of which the first `skip` belong to its neighbour.
struct Cols {
    int64_t at;
    int skip;
    bool on;
};

template <int VE>
__device__ __forceinline__ Cols lane_cols(int64_t slab, int lanes, int lane, int64_t d) {
    Cols c;
    const int64_t c0 = (slab * lanes + lane) * VE;
    c.on = c0 < d;
    c.at = c0 > d - VE ? d - VE : c0;
    c.skip = static_cast<int>(c0 - c.at);
    return c;
}

template <typename TO, int VE>
__device__ __forceinline__ void put_row(const SumArgs &a, int64_t row, const Cols &c,
                                        vec<float, VE> v) {
    if (row >= a.row_cap || !c.on) return;
    TO *p = static_cast<TO *>(a.out) + row * a.ld_out + c.at;
    v *= a.scale;
    if (a.accumulate) v += load_f32<TO, VE>(p);
    if (c.skip == 0) {
        store_f32<TO, VE>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (e >= c.skip) p[e] = static_cast<TO>(v[e]);
    }
}

template <int VE>
__device__ __forceinline__ void put_part(const SumArgs &a, int64_t row, const Cols &c,
                                         vec<float, VE> v) {
    if (!c.on) return;
    store_f32<float, VE>(a.part + row * a.d + c.at, v);   // neighbours store equal values
}

template <typename TI, typename TO, int VE>
__global__ __launch_bounds__(kSumThreads) void k_embedding_sums(SumArgs a) {
    const int per = kSumThreads / a.lanes;
    const int lane = threadIdx.x & (a.lanes - 1);
    if (static_cast<int64_t>(blockIdx.x) >= a.sum_blocks) {
        // zero the rows of the table that no id names: one row per lane group and turn
        const int64_t groups = (static_cast<int64_t>(gridDim.x) - a.sum_blocks) * per;
        int64_t r = (static_cast<int64_t>(blockIdx.x) - a.sum_blocks) * per + threadIdx.x / a.lanes;
        for (; r < a.num_rows; r += groups) {
            if (a.touched[r]) continue;
            TO *p = static_cast<TO *>(a.out) + r * a.ld_out;
            for (int64_t s = 0; s < a.slabs; ++s) {
                const Cols c = lane_cols<VE>(s, a.lanes, lane, a.d);
                if (c.on) store_f32<TO, VE>(p + c.at, vec<float, VE>(0.f));
            }
        }
        return;
    }
    const int64_t g = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / a.lanes;
    const int64_t chunk = g / a.slabs;
    if (chunk >= a.chunks) return;
    const Cols c = lane_cols<VE>(g - chunk * a.slabs, a.lanes, lane, a.d);
    const int64_t e0 = chunk * a.chunk, far = e0 + 2 * a.chunk;
    const int64_t e1 = e0 + a.chunk < a.n ? e0 + a.chunk : a.n;
    const uint32_t none = a.num_rows;
    uint32_t cur = a.key[e0];
    const uint32_t after = e1 < a.n ? a.key[e1] : none;
    const uint32_t after2 = far < a.n ? a.key[far] : none;
    bool earlier = e0 > 0 && a.key[e0 - 1] == cur;       // the first run began in an earlier chunk
    if (cur >= a.num_rows) return;
    int64_t rank = a.chunk_rank ? static_cast<int64_t>(a.chunk_rank[chunk]) : 0;
    const TI *dout = static_cast<const TI *>(a.dout) + (c.on ? c.at : 0);
    typedef typename loose<TI, VE>::type Raw;
    const auto row = [&](uint32_t p) {
        return *reinterpret_cast<const Raw *>(dout + static_cast<int64_t>(p) * a.ld_dout);
    };
    vec<float, VE> acc(0.f);
    bool ended = false;      // reached the positions without a gradient row
    for (int64_t e = e0; e < e1 && !ended; e += kSumUnroll) {
        uint32_t k[kSumUnroll];
        Raw v[kSumUnroll];
        // every load is made (of the chunk's last row beyond its end), so that none waits for a
        // branch
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) {
            const int64_t i = e + u < e1 ? e + u : e1 - 1;
            k[u] = e + u < e1 ? a.key[i] : none;
            v[u] = row(a.pos[i]);
        }
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) {
            if (k[u] >= a.num_rows) {
                ended = true;
                break;
            }
            if (k[u] != cur) {
                if (earlier)
                    put_part<VE>(a, 2 * chunk, c, acc);
                else
                    put_row<TO, VE>(a, a.chunk_rank ? rank : cur, c, acc);
                earlier = false;
                cur = k[u];
                ++rank;
                acc = vec<float, VE>(0.f);
            }
            acc += __builtin_convertvector(v[u], vec<float, VE>);
        }
    }
    if (earlier) {
        put_part<VE>(a, 2 * chunk, c, acc);
    } else if (after == cur) {
        put_part<VE>(a, 2 * chunk + 1, c, acc);
        if (after2 == cur && lane == 0 && g == chunk * a.slabs)     // beyond the next chunk as well
            a.long_runs[1 + atomicAdd(a.long_runs, 1u)] = static_cast<uint32_t>(chunk);
    } else {
        put_row<TO, VE>(a, a.chunk_rank ? rank : cur, c, acc);
    }
}

// The sum over a workgroup's lane groups of their acc, in the groups' order, for the first group; a
// thread adds the groups' values of one column.  Every thread of the workgroup calls it.
template <int VE, int THREADS>
__device__ __forceinline__ void join_groups(vec<float, VE> &acc, float *sm, int lanes) {
    const int t = threadIdx.x;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VE; ++e) sm[e * THREADS + t] = acc[e];
    __syncthreads();
    for (int i = t; i < lanes * VE; i += THREADS) {
        float *p = sm + i / lanes * THREADS + (i & (lanes - 1));
        float x = p[0];
#pragma unroll 8
        for (int g = lanes; g < THREADS; g += lanes) x += p[g];
        p[0] = x;
    }
    __syncthreads();
    if (t < lanes)
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = sm[e * THREADS + t];
}

// Joins the partial sums: a lane group takes a chunk's last run where it ends in the next chunk, and
// the workgroups past sum_blocks take the listed longer runs, whose partial sums their lane
// groups add in turn, and then each other's sums in the groups' order.
template <typename TO, int VE>
__global__ __launch_bounds__(kSumThreads) void k_embedding_join(SumArgs a) {
    __shared__ float sm[kSumThreads * VE];
    const int groups = kSumThreads / a.lanes;
    const int grp = threadIdx.x / a.lanes, lane = threadIdx.x & (a.lanes - 1);
    if (static_cast<int64_t>(blockIdx.x) < a.sum_blocks) {
        const int64_t g = static_cast<int64_t>(blockIdx.x) * groups + grp;
        const int64_t chunk = g / a.slabs;
        const int64_t e0 = chunk * a.chunk, e1 = e0 + a.chunk, far = e1 + a.chunk;
        if (e1 >= a.n) return;
        const uint32_t none = a.num_rows;
        const uint32_t cur = a.key[e1 - 1], after = a.key[e1];
        const uint32_t before = e0 > 0 ? a.key[e0 - 1] : none;
        const uint32_t after2 = far < a.n ? a.key[far] : none;
        if (cur >= none || after != cur || before == cur || after2 == cur) return;
        const Cols c = lane_cols<VE>(g - chunk * a.slabs, a.lanes, lane, a.d);
        if (!c.on) return;
        const float *p = a.part + c.at;
        const vec<float, VE> acc = load_f32<float, VE>(p + (2 * chunk + 1) * a.d) +
                                   load_f32<float, VE>(p + (2 * chunk + 2) * a.d);
        put_row<TO, VE>(a, a.chunk_rank ? static_cast<int64_t>(a.chunk_rank[chunk + 1]) : cur, c, acc);
        return;
    }
    const int64_t b = static_cast<int64_t>(blockIdx.x) - a.sum_blocks;
    const int64_t wide = (static_cast<int64_t>(gridDim.x) - a.sum_blocks) / a.slabs;
    const Cols c = lane_cols<VE>(b % a.slabs, a.lanes, lane, a.d);
    const uint32_t count = *a.long_runs;
    for (uint32_t r = static_cast<uint32_t>(b / a.slabs); r < count; r += static_cast<uint32_t>(wide)) {
        const int64_t chunk = a.long_runs[1 + r];
        const uint32_t cur = a.key[(chunk + 1) * a.chunk];
        // chunks after `chunk` whose first key is cur, a workgroup's width at a time
        int64_t last = chunk;
        for (;;) {
            const int64_t q = last + 1 + threadIdx.x;
            const int in = __syncthreads_count(q < a.chunks && a.key[q * a.chunk] == cur);
            last += in;
            if (in < kSumThreads) break;
        }
        vec<float, VE> acc(0.f);
        if (c.on) {
            const float *p = a.part + c.at;
            if (grp == 0) acc = load_f32<float, VE>(p + (2 * chunk + 1) * a.d);
#pragma unroll 8
            for (int64_t q = chunk + 1 + grp; q <= last; q += groups)
                acc += load_f32<float, VE>(p + 2 * q * a.d);
        }
        join_groups<VE, kSumThreads>(acc, sm, a.lanes);
        // the run's rank is that of the next chunk's first run
        if (grp == 0)
            put_row<TO, VE>(a, a.chunk_rank ? static_cast<int64_t>(a.chunk_rank[chunk + 1]) : cur, c, acc);
    }
}

// ---- few positions --------------------------------------------------------------------------------
//
// With few positions the launches cost more than the work: one
// launch does it all.
//
// The distinct ids: every workgroup sorts all positions for itself, and takes the runs that begin in
// its part of the sorted list.
//
// A dense table: a workgroup owns the rows r with r mod 2^shift = blockIdx.x, so that neighbouring
// frequent ids go to different ones.  It picks its positions from the list of ids, which all read, in
// their order, clears its unnamed rows where the table is written, and sorts its own positions only,
// by the rest of the id.  1024 x 64 fp32 over 10000 rows: 7.6 us a call
// among others (10 under a profiler): the kernel's loading, picking, clearing, sorting and adding, which wait
// for each other behind barriers; a launch's own share is some 2.6.
//
// Both: a lane group adds a short run, all groups together, one after the other, the long ones.
constexpr int kFewThreads = 512;   // (workgroups of 1024 start up to 6 us apart, of 512 half that)
constexpr int kFewRounds = 4;
constexpr int kFewMost = kFewRounds * kFewThreads;
constexpr int kFewShare = 16;      // sorted positions per workgroup
constexpr int kFewRun = 32;        // longest run that one lane group takes
// Dense tables of up to kBucketMid positions, and of up to kBucketMost where a row of dout has at most
// kBucketBytes bytes, go by buckets (all ids of a zipf law: 8192 x 104 bf16 over 50000 rows 23 us for the
// sort's 44, 16384 x 256 over 20000 37 for 44, but 16384 x 400 over 3000 53 for 45: the most frequent
// row's many positions belong to one workgroup).
constexpr int kBucketMid = 16 * kFewThreads, kBucketMost = 32 * kFewThreads;
constexpr int64_t kBucketBytes = 512;
constexpr int kBucketWide = 256;   // workgroups
constexpr int kBucketRows = 16 * kBucketMost / 64;  // of a workgroup: clears_all() is past 16 a position

// The sum of positions pos[i0], pos[i0 + step], ... below pos[end].
template <typename TI, int VE>
__device__ __forceinline__ vec<float, VE> sum_run(const SumArgs &a, const uint16_t *pos, int i0, int end,
                                                  int step, const Cols &c) {
    typedef typename loose<TI, VE>::type Raw;
    const TI *dout = static_cast<const TI *>(a.dout);
    vec<float, VE> acc(0.f);
    for (int i = i0; i < end; i += kSumUnroll * step) {
        Raw v[kSumUnroll];
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) {
            const int at = i + u * step < end ? i + u * step : i;
            v[u] = *reinterpret_cast<const Raw *>(dout + static_cast<int64_t>(pos[at]) * a.ld_dout +
                                                  (c.on ? c.at : 0));
        }
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u)
            if (i + u * step < end) acc += __builtin_convertvector(v[u], vec<float, VE>);
    }
    return acc;
}

// The run that begins at sorted position i and is longer than kFewRun, by the whole workgroup.
template <typename TI, typename TO, int VE>
__device__ __forceinline__ void sum_long(const SumArgs &a, const uint32_t *key, const uint16_t *pos,
                                         int i, int n, int64_t row, int slab, float *sm) {
    const int groups = kFewThreads / a.lanes, grp = threadIdx.x / a.lanes;
    int end = i + kFewRun + 1, over = n;     // the first position of another key
    while (end < over) {
        const int mid = (end + over) / 2;
        if (key[mid] == key[i]) end = mid + 1; else over = mid;
    }
    const Cols c = lane_cols<VE>(slab, a.lanes, threadIdx.x & (a.lanes - 1), a.d);
    vec<float, VE> acc = sum_run<TI, VE>(a, pos, i + grp, end, groups, c);
    join_groups<VE, kFewThreads>(acc, sm, a.lanes);
    if (grp == 0) put_row<TO, VE>(a, row, c, acc);
}

template <typename TI, typename TO, int VE>
__global__ __launch_bounds__(kFewThreads) void k_embedding_few(SortArgs q, SumArgs a) {
    __shared__ OneSort<kFewRounds, kFewThreads> m;
    __shared__ uint32_t sw[kFewThreads / 64];
    __shared__ uint32_t rank_of[kFewShare];
    __shared__ uint32_t long_runs;       // one bit per position of the share
    __shared__ float sm[kFewThreads * VE];
    const int t = threadIdx.x, n = static_cast<int>(q.n);
    const int groups = kFewThreads / a.lanes, grp = t / a.lanes, lane = t & (a.lanes - 1);
    if (t == 0) long_runs = 0;
    uint32_t keys[kFewRounds], pos[kFewRounds];
    load_keys<kFewRounds, kFewThreads>(q, keys);
    own_positions<kFewRounds, kFewThreads>(q.n, pos);
    sort_one(n, q.passes, q.bits, m, keys, pos);
    const int lo = static_cast<int>(blockIdx.x) * kFewShare;
    const auto head = [&](int i) { return is_head(m.key[i], i > 0 ? m.key[i - 1] : 0u, i == 0, q.num_rows); };
    // ranks of the runs; the first workgroup writes the list
    uint32_t carry = 0;
    for (int r0 = 0; r0 < n; r0 += kFewThreads) {
        const int i = r0 + t;
        const uint32_t h = i < n && head(i);
        uint32_t total;
        const uint32_t at = carry + block_exclusive_scan<uint32_t, kFewThreads>(h, &total, sw);
        if (i >= lo && i < lo + kFewShare) rank_of[i - lo] = at;
        if (blockIdx.x == 0 && h && at < q.row_cap) q.uniq[at] = static_cast<int32_t>(m.key[i]);
        carry += total;
    }
    if (blockIdx.x == 0 && t == 0) {
        *q.d_n_uniq = carry;
        if (carry > q.row_cap) set_status(q.status, GNN_ERR_CAPACITY);
    }
    __syncthreads();
    const int hi = lo + kFewShare < n ? lo + kFewShare : n;
    for (int item = grp; item < (hi - lo) * a.slabs; item += groups) {
        const int i = lo + item / a.slabs;
        if (!head(i)) continue;
        if (i + kFewRun < n && m.key[i + kFewRun] == m.key[i]) {
            if (lane == 0) atomicOr(&long_runs, 1u << (i - lo));
            continue;
        }
        int end = i + 1;
        while (end < n && m.key[end] == m.key[i]) ++end;
        const Cols c = lane_cols<VE>(item % a.slabs, a.lanes, lane, a.d);
        put_row<TO, VE>(a, rank_of[i - lo], c, sum_run<TI, VE>(a, m.pos, i, end, 1, c));
    }
    __syncthreads();
    for (uint32_t left = long_runs; left != 0; left &= left - 1) {
        const int i = lo + __ffs(static_cast<int>(left)) - 1;
        for (int slab = 0; slab < a.slabs; ++slab)
            sum_long<TI, TO, VE>(a, m.key, m.pos, i, n, rank_of[i - lo], slab, sm);
    }
}

template <typename TI, typename TO, int VE, int ROUNDS>
__global__ __launch_bounds__(kFewThreads) void k_embedding_buckets(SortArgs q, SumArgs a, int shift,
                                                                   int zero) {
    constexpr int kWaves = kFewThreads / 64, kMost = ROUNDS * kFewThreads;
    __shared__ OneSort<ROUNDS, kFewThreads> m;
    __shared__ uint16_t runs[kMost];     // where runs begin: short ones from the front, long ones from the back
    __shared__ uint32_t found[kWaves], count[2];
    __shared__ float sm[kFewThreads * VE];
    __shared__ uint8_t named[kBucketRows];
    const int t = threadIdx.x, w = t >> 6;
    const int groups = kFewThreads / a.lanes, grp = t / a.lanes, lane = t & (a.lanes - 1);
    const int slab = blockIdx.y;
    const Cols c = lane_cols<VE>(slab, a.lanes, lane, a.d);
    const uint32_t b = blockIdx.x, low = (1u << shift) - 1u;
    const uint64_t below = (1ull << lane_id()) - 1ull;
    const int rounds = (static_cast<int>(q.n) + kFewThreads - 1) / kFewThreads;
    uint32_t keys[ROUNDS], pos[ROUNDS];
    load_keys<ROUNDS, kFewThreads>(q, keys);
    own_positions<ROUNDS, kFewThreads>(q.n, pos);
    if (t < 2) count[t] = 0;
    if (zero)
        for (int i = t; i < kBucketRows; i += kFewThreads) named[i] = 0;
    uint32_t total = 0;
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j)
        if (j < rounds) total += __popcll(__ballot(keys[j] < q.num_rows && (keys[j] & low) == b));
    if (lane_id() == 0) found[w] = total;
    __syncthreads();
    uint32_t at = 0;
    int n = 0;                           // this workgroup's positions
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i < w) at += found[i];
        n += static_cast<int>(found[i]);
    }
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        if (j >= rounds) continue;
        const bool mine = keys[j] < q.num_rows && (keys[j] & low) == b;
        const uint64_t all = __ballot(mine);
        if (mine) {
            const uint32_t to = at + __popcll(all & below);
            m.key[to] = keys[j] >> shift;
            m.pos[to] = static_cast<uint16_t>(pos[j]);
            if (zero) named[keys[j] >> shift] = 1;
        }
        at += __popcll(all);
    }
    __syncthreads();
    if (zero)
        for (uint32_t r = grp; (r << shift) + b < q.num_rows; r += groups) {
            if (named[r] || !c.on) continue;
            store_f32<TO, VE>(static_cast<TO *>(a.out) +
                                  static_cast<int64_t>((r << shift) + b) * a.ld_out + c.at,
                              vec<float, VE>(0.f));
        }
    if (n == 0) return;
    const int mine = (n + kFewThreads - 1) / kFewThreads, i0 = w * 64 * mine + lane_id();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
        if (j >= mine) continue;
        const int i = i0 + j * 64;
        keys[j] = i < n ? m.key[i] : ~0u;        // after every position of the same digits
        pos[j] = i < n ? m.pos[i] : 0u;
    }
    __syncthreads();
    sort_one(n, q.passes, q.bits, m, keys, pos);
    for (int i = t; i < n; i += kFewThreads) {
        if (i > 0 && m.key[i] == m.key[i - 1]) continue;
        if (i + kFewRun < n && m.key[i + kFewRun] == m.key[i])
            runs[kMost - 1 - atomicAdd(&count[1], 1u)] = static_cast<uint16_t>(i);
        else
            runs[atomicAdd(&count[0], 1u)] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    for (int r = grp; r < static_cast<int>(count[0]); r += groups) {
        const int i = runs[r];
        int end = i + 1;
        while (end < n && m.key[end] == m.key[i]) ++end;
        put_row<TO, VE>(a, (static_cast<int64_t>(m.key[i]) << shift) + b, c,
                        sum_run<TI, VE>(a, m.pos, i, end, 1, c));
    }
    for (uint32_t r = 0; r < count[1]; ++r) {
        const int i = runs[kMost - 1 - r];
        sum_long<TI, TO, VE>(a, m.key, m.pos, i, n, (static_cast<int64_t>(m.key[i]) << shift) + b, slab,
                             sm);
    }
}

__global__ __launch_bounds__(256) void k_zero_rows(char *out, int64_t row_bytes, int64_t ld_bytes,
                                                   int64_t rows) {
    // one row per wavefront and turn, 16 bytes a lane, then the row's last 2-byte pieces
    const int lane = lane_id();
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); r < rows;
         r += static_cast<int64_t>(gridDim.x) * 4) {
        char *p = out + r * ld_bytes;
        int64_t b = static_cast<int64_t>(lane) * 16;
        for (; b + 16 <= row_bytes; b += 1024)
            *reinterpret_cast<loose<uint16_t, 8>::type *>(p + b) = vec<uint16_t, 8>(uint16_t(0));
        for (int64_t q = (row_bytes & ~int64_t(15)) + 2 * lane; q < row_bytes; q += 128)
            *reinterpret_cast<uint16_t *>(p + q) = 0;
    }
}

// What the gradient keeps in the workspace.
struct GradSpace {
    uint32_t *key[2], *pos[2], *hist, *heads, *chunk_rank, *long_runs;
    uint8_t *touched;
    float *part;
    int32_t chunk;
    int64_t chunks, touched_words;
    int32_t tiles;
    size_t bytes;
};

// Chunk length: 64 positions, so that the partial sums of a chunk's two ends cost at most a
// sixteenth of its rows of fp32, or shorter where that leaves too few lane groups.
int32_t chunk_for(int64_t n) {
    int64_t c = 64;
    while (c > kChunkMin && n / c < 2048) c /= 2;
    return static_cast<int32_t>(c);
}

// A written dense table: rows that no id names are zeroed by their marks, or, where at most one row in
// 16 can be named, the whole table is cleared first (the rows then written twice are fewer than the
// marks are worth).
bool clears_all(int64_t n, int64_t num_rows) { return n <= num_rows / 16; }

GradSpace carve_grad(int64_t n, int64_t num_rows, int64_t d, char *base) {
    GradSpace g{};
    size_t off = 0;
    auto take = [&](int64_t words) {
        off = (off + 255) & ~static_cast<size_t>(255);
        uint32_t *p = base ? reinterpret_cast<uint32_t *>(base + off) : nullptr;
        off += static_cast<size_t>(words < 1 ? 1 : words) * 4;
        return p;
    };
    g.chunk = chunk_for(n);
    g.chunks = (n + g.chunk - 1) / g.chunk;
    g.tiles = static_cast<int32_t>((n + kSortTile - 1) / kSortTile);
    g.touched_words = (num_rows + 3) / 4;
    for (int i = 0; i < 2; ++i) {
        g.key[i] = take(n);
        g.pos[i] = take(n);
    }
    g.hist = take(static_cast<int64_t>(g.tiles + 1) * kDigits);
    g.heads = take(g.tiles);
    g.chunk_rank = take(g.chunks);
    g.long_runs = take(1 + g.chunks);
    g.touched = reinterpret_cast<uint8_t *>(take(clears_all(n, num_rows) ? 0 : g.touched_words));
    g.part = reinterpret_cast<float *>(take(2 * g.chunks * d));
    g.bytes = off;
    return g;
}

template <typename TI, typename TO, int VE>
hipError_t run_sums(const EmbedGradArgs &a, const GradSpace &g, const SortArgs &sort,
                    const uint32_t *key, const uint32_t *pos, bool zero_untouched, hipStream_t s) {
    SumArgs p{};
    p.key = key;
    p.pos = pos;
    p.n = a.n;
    p.num_rows = static_cast<uint32_t>(a.num_rows);
    p.dout = a.dout;
    p.ld_dout = a.ld_dout;
    p.d = a.d;
    p.scale = a.scale;
    p.out = a.out;
    p.ld_out = a.ld_out;
    p.accumulate = a.accumulate;
    p.chunk_rank = a.rows ? g.chunk_rank : nullptr;
    p.row_cap = a.rows ? a.row_cap : a.num_rows;
    p.part = g.part;
    p.long_runs = g.long_runs;
    p.chunk = g.chunk;
    p.chunks = g.chunks;
    const int64_t cpr = (a.d + VE - 1) / VE;
    p.lanes = 1;
    while (p.lanes < cpr && p.lanes < 64) p.lanes *= 2;
    p.slabs = static_cast<int32_t>((cpr + p.lanes - 1) / p.lanes);
    if (key == nullptr && a.rows) {
        hipLaunchKernelGGL((k_embedding_few<TI, TO, VE>),
                           dim3(static_cast<unsigned>((a.n + kFewShare - 1) / kFewShare)),
                           dim3(kFewThreads), 0, s, sort, p);
        return hipGetLastError();
    }
    if (key == nullptr) {
        int shift = 6;
        while (p.slabs << shift < kBucketWide && ((a.n * p.lanes) >> shift) > kFewThreads) ++shift;
        SortArgs q = sort;
        int nb = 1;
        while ((static_cast<uint64_t>(a.num_rows - 1) >> shift >> nb) != 0) ++nb;
        q.passes = (nb + kSortBits - 1) / kSortBits;
        q.bits = (nb + q.passes - 1) / q.passes;
        const dim3 grid(1u << shift, static_cast<unsigned>(p.slabs)), block(kFewThreads);
        const int zero = zero_untouched ? 1 : 0;
        if (a.n <= kFewMost)
            hipLaunchKernelGGL((k_embedding_buckets<TI, TO, VE, kFewRounds>), grid, block, 0, s, q, p,
                               shift, zero);
        else if (a.n <= kBucketMid)
            hipLaunchKernelGGL((k_embedding_buckets<TI, TO, VE, kBucketMid / kFewThreads>), grid, block,
                               0, s, q, p, shift, zero);
        else
            hipLaunchKernelGGL((k_embedding_buckets<TI, TO, VE, kBucketMost / kFewThreads>), grid, block, 0, s, q, p,
                               shift, zero);
        return hipGetLastError();
    }
    const int per = kSumThreads / p.lanes;
    p.sum_blocks = (g.chunks * p.slabs + per - 1) / per;
    int64_t zero_blocks = 0;
    if (zero_untouched) {
        p.touched = g.touched;
        zero_blocks = (a.num_rows + per * 8 - 1) / (per * 8);
        if (zero_blocks > 16384) zero_blocks = 16384;
    }
    if (p.sum_blocks + zero_blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((k_embedding_sums<TI, TO, VE>),
                       dim3(static_cast<unsigned>(p.sum_blocks + zero_blocks)), dim3(kSumThreads),
                       0, s, p);
    if (g.chunks > 1) {
        // a listed run holds a whole chunk
        const int64_t most = g.chunks / 2 < kJoinRuns ? g.chunks / 2 : kJoinRuns;
        hipLaunchKernelGGL((k_embedding_join<TO, VE>),
                           dim3(static_cast<unsigned>(p.sum_blocks + most * p.slabs)),
                           dim3(kSumThreads), 0, s, p);
    }
    return hipGetLastError();
}

template <typename TI, typename TO>
hipError_t pick_sums(const EmbedGradArgs &a, const GradSpace &g, const SortArgs &q, const uint32_t *key,
                     const uint32_t *pos, bool zero, hipStream_t s) {
    constexpr int kWide = sizeof(TI) == 2 ? 8 : 4;      // 16 bytes of dout a lane
    if (a.d >= kWide) return run_sums<TI, TO, kWide>(a, g, q, key, pos, zero, s);
    return run_sums<TI, TO, 1>(a, g, q, key, pos, zero, s);
}

}  // namespace

hipError_t launch_embedding_lookup(LookupArgs a, hipStream_t s) {
    if (a.n <= 0) return hipSuccess;
    if (a.table_type == GNN_F32)
        return a.out_type == GNN_F32 ? pick_lookup<float, float>(a, s) : pick_lookup<float, bf16>(a, s);
    return a.out_type == GNN_F32 ? pick_lookup<bf16, float>(a, s) : pick_lookup<bf16, bf16>(a, s);
}

size_t embedding_grad_bytes(int64_t n, int64_t num_rows, int64_t d) {
    return carve_grad(n, num_rows, d, nullptr).bytes;
}

hipError_t launch_embedding_grad(const EmbedGradArgs &a, hipStream_t s) {
    const int elem = a.out_type == GNN_F32 ? 4 : 2;
    const bool dense = !a.rows;
    const bool written = dense && !a.accumulate;
    const bool clear_all = written && clears_all(a.n, a.num_rows);
    if (clear_all) {
        const int64_t blocks = (a.num_rows + 15) / 16;
        hipLaunchKernelGGL(k_zero_rows, dim3(static_cast<unsigned>(blocks < 32768 ? blocks : 32768)),
                           dim3(256), 0, s, static_cast<char *>(a.out), a.d * elem, a.ld_out * elem,
                           a.num_rows);
    }
    if (a.n == 0 && (!written || clear_all) && dense) return hipGetLastError();
    const GradSpace g = carve_grad(a.n, a.num_rows, a.d, a.ws);
    SortArgs q{};
    q.ids = a.ids;
    q.d_n = a.d_n;
    q.n = a.n;
    q.pad_id = a.pad_id;
    q.num_rows = static_cast<uint32_t>(a.num_rows);
    q.status = a.status;
    q.hist = g.hist;
    q.tiles = g.tiles;
    q.scanned = g.tiles > kSumTiles;
    if (written && !clear_all) {
        q.touched = g.touched;
        q.touched_words = g.touched_words;
    }
    int nb = 1;
    while ((static_cast<uint64_t>(a.num_rows) >> nb) != 0) ++nb;
    q.passes = (nb + kSortBits - 1) / kSortBits;
    q.bits = (nb + q.passes - 1) / q.passes;
    q.uniq = a.uniq;
    q.d_n_uniq = a.d_n_uniq;
    q.row_cap = a.row_cap;
    q.chunk_rank = g.chunk_rank;
    q.chunk = g.chunk;
    const uint32_t *key, *pos;
    q.long_runs = g.long_runs;
    const int64_t row = a.d * (a.dout_type == GNN_F32 ? 4 : 2);
    const int64_t few = a.rows ? kFewMost : row <= kBucketBytes ? kBucketMost : kBucketMid;
    if (a.n > 0 && a.n <= few) {
        key = pos = nullptr;        // sorted by the kernel that adds
    } else if (a.n <= kOneTile) {
        q.key_out = g.key[0];
        q.pos_out = g.pos[0];
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kOneThreads), 0, s, q);
        key = g.key[0];
        pos = g.pos[0];
    } else {
        for (int p = 0; p < q.passes; ++p) {
            q.shift = p * q.bits;
            q.key_in = p ? g.key[(p + 1) & 1] : nullptr;
            q.pos_in = p ? g.pos[(p + 1) & 1] : nullptr;
            q.key_out = g.key[p & 1];
            q.pos_out = g.pos[p & 1];
            const dim3 grid(static_cast<unsigned>(g.tiles));
            hipLaunchKernelGGL(k_sort_count, grid, dim3(kSortThreads), 0, s, q);
            if (q.scanned) hipLaunchKernelGGL(k_sort_scan, dim3(kDigits), dim3(256), 0, s, q);
            hipLaunchKernelGGL(k_sort_place, grid, dim3(kSortThreads), 0, s, q);
        }
        key = g.key[(q.passes - 1) & 1];
        pos = g.pos[(q.passes - 1) & 1];
        if (!dense) {
            HeadArgs h{};
            h.key = key;
            h.n = a.n;
            h.num_rows = q.num_rows;
            h.heads = g.heads;
            h.tiles = g.tiles;
            h.uniq = a.uniq;
            h.d_n_uniq = a.d_n_uniq;
            h.row_cap = a.row_cap;
            h.chunk_rank = g.chunk_rank;
            h.chunk = g.chunk;
            h.status = a.status;
            const dim3 grid(static_cast<unsigned>(g.tiles));
            hipLaunchKernelGGL(k_count_heads, grid, dim3(kSortThreads), 0, s, h);
            hipLaunchKernelGGL(k_emit_heads, grid, dim3(kSortThreads), 0, s, h);
        }
    }
    const bool zero = written && !clear_all;
    if (a.dout_type == GNN_F32)
        return a.out_type == GNN_F32 ? pick_sums<float, float>(a, g, q, key, pos, zero, s)
                                     : pick_sums<float, bf16>(a, g, q, key, pos, zero, s);
    return a.out_type == GNN_F32 ? pick_sums<bf16, float>(a, g, q, key, pos, zero, s)
                                 : pick_sums<bf16, bf16>(a, g, q, key, pos, zero, s);
}

}  // namespace gnnmb
