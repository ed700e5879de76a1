// Launchers of the learned side of the path (embedding lookup and gradient, cross attention,
// orthogonalised updates), and the element types they share.  Internal; not part of the ABI.
#pragma once

#include "common.hpp"

namespace gnnmb {

typedef __bf16 bf16;

template <typename T, int N>
using vec = T __attribute__((ext_vector_type(N)));
// The same vector at any address that is aligned for one element: global loads and stores of gfx950
// need no more than the element's alignment.
template <typename T, int N>
struct loose {
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <typename T, int N>
__device__ __forceinline__ vec<float, N> load_f32(const T *p) {
    const typename loose<T, N>::type v = *reinterpret_cast<const typename loose<T, N>::type *>(p);
    return __builtin_convertvector(v, vec<float, N>);
}

// Rounds to nearest even where T is bf16.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T *p, vec<float, N> v) {
    *reinterpret_cast<typename loose<T, N>::type *>(p) = __builtin_convertvector(v, vec<T, N>);
}

// A grid has fewer than 2^32 threads a dimension: launch(first, blocks) enqueues `blocks` workgroups of
// `threads` from the first on, in as many pieces as that takes (one, but for calls of gigabytes).
template <typename F>
hipError_t launch_pieces(int64_t blocks, int threads, F launch) {
    const int64_t most = (int64_t(1) << 31) / threads;
    for (int64_t first = 0; first < blocks; first += most) {
        launch(first, static_cast<unsigned>(blocks - first < most ? blocks - first : most));
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// ---- embedding ----------------------------------------------------------------------------------

struct LookupArgs {
    const void *table;
    int32_t table_type, out_type;
    int64_t num_rows, d, ld;
    const int32_t *ids;
    const int64_t *d_n;
    int64_t n;
    float scale;
    int32_t pad_id;
    void *out;
    int64_t ld_out;
    int32_t *status;
    uint32_t cpr;       // vectors per row (set by the launcher, with its divisor)
    FastDiv by_cpr;
    int64_t first_block;
};
hipError_t launch_embedding_lookup(LookupArgs a, hipStream_t s);

struct EmbedGradArgs {
    const int32_t *ids;
    const int64_t *d_n;
    int64_t n;
    const void *dout;
    int32_t dout_type, out_type;
    int64_t ld_dout;
    float scale;
    int32_t pad_id;
    int64_t num_rows, d;
    void *out;              // dense: [num_rows, ld_out]; rows: [row_cap, ld_out]
    int64_t ld_out;
    int32_t accumulate;     // dense only
    int32_t rows;           // 1: the rows form, 0: dense
    int32_t *uniq;          // rows: [row_cap] distinct ids, ascending
    int64_t *d_n_uniq;
    int64_t row_cap;
    int32_t *status;
    char *ws;
};
// Bytes of workspace that launch_embedding_grad needs for these sizes.
size_t embedding_grad_bytes(int64_t n, int64_t num_rows, int64_t d);
hipError_t launch_embedding_grad(const EmbedGradArgs &a, hipStream_t s);

// ---- cross attention ------------------------------------------------------------------------------

struct AttendArgs {
    int32_t type, heads, kv, group, d;     // group = heads / kv
    int64_t n_seq, n_q, n_k, max_q, max_k;
    float scale, scale2;                   // scale2 = scale * log2(e)
    const int32_t *q_indptr, *k_indptr;
    const int64_t *k_count;
    const void *q, *k, *v;
    int64_t ld_q, ld_k, ld_v;
    void *out;                             // backward: read
    int64_t ld_out;
    float *lse;                            // [n_q, heads]; backward: read
    int32_t *status;
    // backward
    const void *dout;
    int64_t ld_dout;
    void *dq, *dk, *dv;
    int64_t ld_dq, ld_dk, ld_dv;
    // set by the launcher
    FastDiv by_group;
    int64_t first_block;
    int32_t splits;
    int64_t per;           // states (or rows) per split
    char *ws;
    float2 *stat;          // [n_q * heads] {lse log2(e), dout . out}
    float *part;           // partial sums of the splits
    float2 *part_stat;     // [splits, n_q * heads] {maximum, sum}
};
size_t attend_bytes(const AttendArgs &a, bool backward);
hipError_t launch_attend(AttendArgs a, bool backward, char *ws, hipStream_t s);

// ---- orthogonalised updates -----------------------------------------------------------------------

struct NewtonArgs {
    const void *g;          // [batch][rows, ld_g]
    int32_t type;
    int64_t rows, cols, ld_g, batch, batch_g;
    int32_t steps;
    float coefs[3];
    float eps, scale;
    void *out;              // [batch][rows, ld_out], g's type
    int64_t ld_out, batch_out;
    char *ws;
};
size_t newton_bytes(int64_t rows, int64_t cols, int64_t batch, int32_t type);
// Whether the values of these steps fit the planes they are kept in.
bool newton_in_range(const float *coefs, int steps);
hipError_t launch_newton(const NewtonArgs &a, hipStream_t s);

}  // namespace gnnmb
