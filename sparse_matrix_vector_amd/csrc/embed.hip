// Rows of a table by token id, and the table's gradient, on gfx950.
//
// With P the tokens x vocabulary 0/1 matrix of the ids, the lookup is
// y = a P E and the gradient dE = a P^T dy: a CSR product whose rows are the
// runs of equal ids among the sorted tokens.  Both stream rows and are bound by
// HBM; the gradient's largest part is writing the table.
//
// Measured, with what the bytes take at the rate of a large copy (5.2 TB/s): 16384 rows
// of 2048 of a table of 50000, fp16 to fp32, 25 us (30); the gradient of 8191 rows of 2048
// in bf16, for 50000 rows of fp32, 97 us (85): 60 for writing the table beside the sort,
// 22 for the sums, 7 for the runs that cross blocks; of 1001 rows of 1111 in fp32 17 us (2):
// three launches that wait for each other, 6.5 + 7.8 + 3.5.
//
// The sort is stable and the sums are added in the order of the tokens within
// fixed blocks of sorted positions: the same bits on every call, no atomics.
#include "elem.hpp"

#include <algorithm>

namespace spmv {
namespace {

// ---------------------------------------------------------------------------
// Lookup: a wave moves one piece of a token's row, 16 bytes of the result per lane
// and access, so that every store of a wave fills whole cache lines (the last
// access of a row starts early where the width is no multiple of it).  16384 rows of
// 2048, fp16 to fp32: 25 us, 6.3 TB/s (52 with 16 bytes of the table per lane, whose
// fp32 results fill lines in two stores); 61 rows: 3.2 us, one chain of two loads.
// ---------------------------------------------------------------------------
// N elements at any element's address.
template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_row(const typename E::T *p) {
    if constexpr (sizeof(Vec<E, N>) == 16) {
        return load_any<E, N>(p);
    } else {
        Vec<E, N> v;
        __builtin_memcpy(&v, __builtin_assume_aligned(p, sizeof(typename E::T)), sizeof v);
        return v;
    }
}

template <typename E, typename Y, int VEC>
__global__ __launch_bounds__(256) void k_embed_lookup(int n_tok, int n_vocab, int dim, int pieces,
                                                      const int *__restrict__ ids,
                                                      const typename E::T *__restrict__ table, int64_t ldt, float scale,
                                                      typename Y::T *__restrict__ y, int64_t ldy) {
    constexpr int U = 4, COLS = 64 * VEC * U;
    const int lane = __lane_id();
    const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tok = (int)(id / pieces), piece = (int)(id - (int64_t)tok * pieces);
    if (tok >= n_tok) return;
    const int row = ids[tok];
    const bool known = (unsigned)row < (unsigned)n_vocab;
    const typename E::T *src = table + (int64_t)(known ? row : 0) * ldt;
    typename Y::T *dst = y + (int64_t)tok * ldy;
    const int c0 = piece * COLS + lane * VEC;
    Vec<E, VEC> v[U];
    if (known) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_row<E, VEC>(src + min(c0 + u * 64 * VEC, dim - VEC));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * VEC;
        if (c >= dim) continue;
        typename Y::T *d = dst + min(c, dim - VEC);
        Vec<Y, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.v[i] = (typename Y::T)(known ? scale * (float)v[u].v[i] : 0.0f);
        store_once<Y, VEC>(d, o);
    }
}

// ---------------------------------------------------------------------------
// The tokens in the order of their ids: sorted[i] the i-th id (n_vocab for ids
// outside the vocabulary, which come last), order[i] its token.
// ---------------------------------------------------------------------------
// Tokens that are ranked by comparing each with all, in one launch, against the digit
// sort's three for every 8 bits of the ids: 1001 tokens 6 us, 8191 tokens 17, 16384
// tokens 28, where ids of 16 bits take 25 by digits (23 for few tokens).
constexpr int ER_ONE = 16384;
constexpr int ER_CHUNK = 4096;       // tokens of a workgroup in the digit sort
constexpr int ER_BITS = 8;
constexpr int ER_BINS = 1 << ER_BITS;
constexpr int ER_MAX_TOK = 1 << 22;

__device__ __forceinline__ int id_key(int id, int n_vocab) { return (int)min((unsigned)id, (unsigned)n_vocab); }

// The gradient's table is cleared beside the sort, by workgroups of the sort's first
// launch that have no part in it: writing the table takes longer than sorting, and
// the rows that have tokens are few.
constexpr int EG_CLEAR = 16384;      // numbers that a workgroup clears
struct Fill {
    float *table;
    int64_t ld, rows;
    int dim, first, blocks;       // the first of those workgroups, and how many there are
};
__device__ __forceinline__ void clear_rows(const Fill &f) {
    const int64_t blk = (int)blockIdx.x - f.first;
    if (f.ld == f.dim || f.rows <= 1) {
        // EG_CLEAR numbers for a workgroup, one after another
        const int64_t n = f.rows * f.dim, from = blk * EG_CLEAR, to = min(n, from + EG_CLEAR);
        for (int64_t i = from + 4 * (int64_t)threadIdx.x; i < to; i += 4096) {
            if (i + 4 <= to)
                store_any<F32, 4>(f.table + i, Vec<F32, 4>{{0.0f, 0.0f, 0.0f, 0.0f}});
            else
                for (int64_t k = i; k < to; ++k) f.table[k] = 0.0f;
        }
    } else {
        // a wave clears a row at a time
        for (int64_t r = blk * 16 + threadIdx.x / 64; r < f.rows; r += (int64_t)f.blocks * 16)
            for (int c = (int)(threadIdx.x % 64); c < f.dim; c += 64) f.table[r * f.ld + c] = 0.0f;
    }
}

// A token's place is the number of tokens with a smaller id, or with its id and
// before it.  A workgroup ranks 64 tokens, and its waves compare them with a part
// of all tokens each; the other side of a comparison is the same for all lanes.
__global__ __launch_bounds__(1024) void k_embed_rank(int n_tok, int n_vocab, const int *__restrict__ ids,
                                                     int *__restrict__ sorted, int *__restrict__ order, Fill fill) {
    __shared__ int count[16][64];
    if ((int)blockIdx.x >= fill.first) {
        clear_rows(fill);
        return;
    }
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int t0 = blockIdx.x * 64, t = t0 + lane;
    const int key = id_key(ids[min(t, n_tok - 1)], n_vocab);
    const int per = (n_tok + 15) / 16;
    const int a = min(wv * per, n_tok), b = min(a + per, n_tok);
    int c = 0;
    // tokens before the 64 count if their id is at most the lane's, those after if it is
    // smaller, that is, at most the lane's less 1; 16 ids at a time, in scalar registers
    auto at_most = [&](int from, int to, int limit) {
        int i = from;
        int k[16], next[16];
        if (i + 16 <= to) {
#pragma unroll
            for (int j = 0; j < 16; ++j) next[j] = ids[i + j];
        }
        for (; i + 16 <= to; i += 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) k[j] = next[j];
            const int ahead = min(i + 16, n_tok - 16);               // there are 16 at least
#pragma unroll
            for (int j = 0; j < 16; ++j) next[j] = ids[ahead + j];
#pragma unroll
            for (int j = 0; j < 16; ++j) c += id_key(k[j], n_vocab) <= limit;
        }
        for (; i < to; ++i) c += id_key(ids[i], n_vocab) <= limit;
    };
    const int b1 = max(a, min(b, t0)), a2 = min(b, max(a, t0 + 64));
    at_most(a, b1, key);
    for (int i = b1; i < a2; ++i) c += id_key(ids[i], n_vocab) <= (i < t ? key : key - 1);
    at_most(a2, b, key - 1);
    count[wv][lane] = c;
    __syncthreads();
    if (wv == 0 && t < n_tok) {
        int at = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) at += count[w][lane];
        sorted[at] = key;
        order[at] = t;
    }
}

// More tokens: a stable sort by digits of 8 bits, lowest first.  counts[digit][chunk].
template <bool FIRST>
__global__ __launch_bounds__(1024) void k_embed_count(int n_tok, int n_vocab, int shift, int chunks,
                                                      const int *__restrict__ keys, int *__restrict__ counts, Fill fill) {
    __shared__ int hist[ER_BINS];
    if ((int)blockIdx.x >= fill.first) {
        clear_rows(fill);
        return;
    }
    if (threadIdx.x < ER_BINS) hist[threadIdx.x] = 0;
    __syncthreads();
    const int s0 = blockIdx.x * ER_CHUNK, s1 = min(n_tok, s0 + ER_CHUNK);
    for (int s = s0 + threadIdx.x; s < s1; s += 1024) {
        const int k = FIRST ? id_key(keys[s], n_vocab) : keys[s];
        atomicAdd(&hist[(k >> shift) & (ER_BINS - 1)], 1);
    }
    __syncthreads();
    if (threadIdx.x < ER_BINS) counts[(size_t)threadIdx.x * chunks + blockIdx.x] = hist[threadIdx.x];
}

// counts becomes its exclusive running sum, in place; one workgroup.
__global__ __launch_bounds__(1024) void k_embed_scan(int n, int *__restrict__ counts) {
    __shared__ int wave_total[16];
    const int lane = __lane_id(), wv = threadIdx.x / 64;
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += 1024) {
        const int i = i0 + threadIdx.x;
        const int v = i < n ? counts[i] : 0;
        const int incl = wave_inclusive_scan(v);
        if (lane == 63) wave_total[wv] = incl;
        __syncthreads();
        int before = base, total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wv) before += wave_total[w];
            total += wave_total[w];
        }
        if (i < n) counts[i] = before + incl - v;
        base += total;
        __syncthreads();
    }
}

template <bool FIRST>
__global__ __launch_bounds__(1024) void k_embed_scatter(int n_tok, int n_vocab, int shift, int chunks,
                                                        const int *__restrict__ keys, const int *__restrict__ from,
                                                        const int *__restrict__ counts, int *__restrict__ keys_out,
                                                        int *__restrict__ order) {
    __shared__ int at[16][ER_BINS];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    for (int i = threadIdx.x; i < 16 * ER_BINS; i += 1024) (&at[0][0])[i] = 0;
    __syncthreads();
    constexpr int PER = ER_CHUNK / 16;
    const int s0 = min(n_tok, (int)blockIdx.x * ER_CHUNK + wv * PER), s1 = min(n_tok, s0 + PER);
    for (int s = s0 + lane; s < s1; s += 64) {
        const int k = FIRST ? id_key(keys[s], n_vocab) : keys[s];
        atomicAdd(&at[wv][(k >> shift) & (ER_BINS - 1)], 1);
    }
    __syncthreads();
    if (threadIdx.x < ER_BINS) {
        int run = counts[(size_t)threadIdx.x * chunks + blockIdx.x];
        for (int w = 0; w < 16; ++w) {
            const int c = at[w][threadIdx.x];
            at[w][threadIdx.x] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int s = s0; s < s1; s += 64) {                // uniform: every lane takes part in the ballots
        const bool in = s + lane < s1;
        const int k = in ? (FIRST ? id_key(keys[s + lane], n_vocab) : keys[s + lane]) : 0;
        const int d = (k >> shift) & (ER_BINS - 1);
        unsigned long long same = __ballot(in);
#pragma unroll
        for (int b = 0; b < ER_BITS; ++b) {
            const unsigned long long ones = __ballot((d >> b) & 1);
            same &= ((d >> b) & 1) ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int lead = in ? __ffsll(same) - 1 : lane;
        int p = 0;
        if (in && lane == lead) p = atomicAdd(&at[wv][d], __popcll(same));
        p = __shfl(p, lead) + rank;
        if (in) {
            keys_out[p] = k;
            order[p] = FIRST ? s + lane : from[s + lane];
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient.  Blocks of `per` sorted positions: a run of equal ids that lies in
// one block is summed and stored there; the parts of a run that crosses blocks
// go to head[block] (the run began before the block) or tail[block] (it begins in
// it) and are added by k_embed_join.  16 rows are on their way for a wave; blocks of 16
// positions, more only past 65536 tokens, so that a training batch has thousands of waves:
// 8191 rows of 2048 in bf16 are 34 MB read, and the sums stored, in 22 us; 1001 rows
// of 1111 in fp32 take 7.8, the chain ids, tokens, rows.
// ---------------------------------------------------------------------------
constexpr int EG_MIN = 16;           // sorted positions of a block at least
constexpr int EG_BLOCKS = 4096;      // blocks at most
constexpr int EJ_WAVES = 8;

// d[0 .. VEC) (+)= scale * v; the first `skip` elements, which the lane before has, are left out.
template <int VEC>
__device__ __forceinline__ void add_row(float *d, const float (&v)[VEC], int skip, float scale, bool add) {
    if (VEC == 1 || skip > 0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i >= skip) d[i] = add ? fmaf(scale, v[i], d[i]) : scale * v[i];
    } else {
#pragma unroll
        for (int p = 0; p < VEC; p += 4) {
            Vec<F32, 4> o, old;
            if (add) old = load_any<F32, 4>(d + p);
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[i] = add ? fmaf(scale, v[p + i], old.v[i]) : scale * v[p + i];
            store_any<F32, 4>(d + p, o);
        }
    }
}

template <typename E, int VEC>
__global__ __launch_bounds__(256) void k_embed_sum(int n_tok, int n_vocab, int dim, int per, int n_blocks, int pieces,
                                                   const int *__restrict__ sorted, const int *__restrict__ order,
                                                   const typename E::T *__restrict__ dy, int64_t lddy, float scale,
                                                   bool add, float *__restrict__ table, int64_t ldt,
                                                   float *__restrict__ heads) {
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t id = (int64_t)blockIdx.x * 4 + wv;
    if (id >= (int64_t)n_blocks * pieces) return;
    const int blk = (int)(id / pieces), piece = (int)(id - (int64_t)blk * pieces);
    const int c = (piece * 64 + lane) * VEC, at = min(c, dim - VEC);
    const bool in = c < dim;
    const int p0 = blk * per, p1 = min(n_tok, p0 + per);
    const typename E::T *src = dy + at;
    constexpr int U = 16;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    bool begun = p0 > 0 && sorted[p0 - 1] == sorted[p0];           // the run began before the block
    for (int q0 = p0; q0 < p1; q0 += 64) {
        // a lane holds one of 64 positions: its id, its token, whether its run ends there
        const int q = min(q0 + lane, n_tok - 1);
        const int key = sorted[q], tok = order[q];
        const int after = q + 1 < n_tok ? sorted[q + 1] : -1;
        const unsigned long long last = __ballot(after != key);
        // ids outside the vocabulary come last, and their rows are not read
        const int n = __popcll(__ballot(q0 + lane < p1 && key < n_vocab));
        for (int j = 0; j < n; j += U) {
            Vec<E, VEC> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = __builtin_amdgcn_readlane(tok, min(j + u, n - 1));
                v[u] = load_row<E, VEC>(src + t * lddy);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j + u >= n) break;
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += (float)v[u].v[i];
                const bool ends = (last >> (j + u)) & 1;
                if (!ends && q0 + j + u + 1 < p1) continue;
                if (in) {
                    if (begun || !ends) {
                        float *d = heads + ((int64_t)(begun ? 0 : n_blocks) + blk) * dim + at;
                        add_row<VEC>(d, acc, c - at, 1.0f, false);
                    } else {
                        const int64_t row = __builtin_amdgcn_readlane(key, j + u);
                        add_row<VEC>(table + row * ldt + at, acc, c - at, scale, add);
                    }
                }
                begun = false;
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
            }
        }
    }
}

// The first position past the run of `key` in sorted[lo .. n), by the whole wave.
__device__ __forceinline__ int run_end(const int *__restrict__ sorted, int lo, int n, int key) {
    int hi = n;
    while (lo < hi) {
        const int s = (hi - lo + 63) / 64;
        const int64_t i = (int64_t)lo + (int64_t)(__lane_id() + 1) * s - 1;
        const int c = __popcll(__ballot(i < hi && sorted[min(i, (int64_t)n - 1)] <= key));
        lo = min(hi, lo + c * s);
        hi = min(hi, lo + s - 1);
    }
    return lo;
}

// The sum of a run that crosses blocks, from the block that it begins in: its
// tail, and the heads of the blocks after it, every EJ_WAVES-th by one wave.
template <int VEC>
__global__ __launch_bounds__(64 * EJ_WAVES) void k_embed_join(int n_tok, int n_vocab, int dim, int per, int n_blocks,
                                                              const int *__restrict__ sorted, float scale, bool add,
                                                              float *__restrict__ table, int64_t ldt,
                                                              const float *__restrict__ heads) {
    constexpr int U = 8;
    __shared__ float part[EJ_WAVES][64 * VEC];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blk = blockIdx.x, p0 = blk * per, p1 = p0 + per;
    if (p1 >= n_tok) return;
    const int key = sorted[p1];
    if (key >= n_vocab || sorted[p1 - 1] != key || (p0 > 0 && sorted[p0 - 1] == key)) return;
    const int c = ((int)blockIdx.y * 64 + lane) * VEC, at = min(c, dim - VEC);
    const int last = (run_end(sorted, p1, n_tok, key) - 1) / per;       // the block that the run ends in
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    if (wv == 0) {
        const Vec<F32, VEC> v = load_row<F32, VEC>(heads + ((int64_t)n_blocks + blk) * dim + at);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = v.v[i];
    }
    for (int b0 = blk + 1 + wv; b0 <= last; b0 += U * EJ_WAVES) {
        Vec<F32, VEC> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load_row<F32, VEC>(heads + (int64_t)min(b0 + u * EJ_WAVES, last) * dim + at);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (b0 + u * EJ_WAVES <= last) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += v[u].v[i];
            }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[wv][lane * VEC + i] = acc[i];
    __syncthreads();
    if (wv == 0 && c < dim) {
        for (int w = 1; w < EJ_WAVES; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += part[w][lane * VEC + i];
        add_row<VEC>(table + (int64_t)key * ldt + at, acc, c - at, scale, add);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
spmv_status check_table(int64_t n_tok, int64_t n_vocab, int64_t dim, int32_t dtype) {
    if (n_tok < 0 || n_vocab < 0 || dim < 0) return fail(SPMV_ERR_INVALID_VALUE, "negative size");
    if (!dtype_ok(dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", dtype);
    return SPMV_OK;
}

int64_t per_block(int64_t n_tok) { return std::max<int64_t>(EG_MIN, ceil_div(n_tok, EG_BLOCKS)); }

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// The workspace's parts: sorted, order (twice where digits are sorted), counts, heads and tails.
struct Parts {
    size_t ints, counts, heads, total;
    bool digits;
    int chunks;
};
Parts parts_of(int64_t n_tok, int64_t dim) {
    Parts p;
    p.digits = n_tok > ER_ONE;
    p.chunks = (int)ceil_div(n_tok, ER_CHUNK);
    p.ints = round256((size_t)n_tok * 4);
    p.counts = p.digits ? round256((size_t)p.chunks * ER_BINS * 4) : 0;
    const int64_t per = per_block(n_tok), blocks = ceil_div(n_tok, per);
    p.heads = blocks > 1 ? (size_t)blocks * 2 * dim * 4 : 0;
    p.total = p.ints * (p.digits ? 4 : 2) + p.counts + round256(p.heads);
    return p;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status embed_lookup(int32_t n_tok, int32_t n_vocab, int32_t dim, int32_t dtype, const int32_t *ids,
                                    const void *table, int64_t ldt, float scale, void *y, int32_t y_dtype, int64_t ldy,
                                    void *stream) {
    spmv_status st = check_table(n_tok, n_vocab, dim, dtype);
    if (st != SPMV_OK) return st;
    if (!dtype_ok(y_dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", y_dtype);
    if (y_dtype != SPMV_F32 && y_dtype != dtype) return fail(SPMV_ERR_UNSUPPORTED, "y must be fp32 or have the table's type");
    if (ldt < dim || ldy < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_tok == 0 || dim == 0) return SPMV_OK;
    if (!ids || !y || (n_vocab > 0 && !table)) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    auto run = [&](auto e, auto t, auto vec) -> spmv_status {
        typedef decltype(e) E;
        typedef decltype(t) Y;
        constexpr int VEC = decltype(vec)::value;
        const int64_t pieces = ceil_div(dim, 64 * VEC * 4), blocks = ceil_div(n_tok * pieces, 4);
        const spmv_status s = check_grid(blocks);
        if (s != SPMV_OK) return s;
        k_embed_lookup<E, Y, VEC><<<(int)blocks, 256, 0, as_stream(stream)>>>(
            n_tok, n_vocab, dim, (int)pieces, ids, static_cast<const typename E::T *>(table), ldt, scale,
            static_cast<typename Y::T *>(y), ldy);
        SPMV_LAUNCHED("k_embed_lookup");
        return SPMV_OK;
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    if (dtype == SPMV_F32) return dim >= 4 ? run(F32{}, F32{}, four) : run(F32{}, F32{}, one);
    auto half = [&](auto e) {
        typedef decltype(e) E;
        if (y_dtype == SPMV_F32) return dim >= 4 ? run(E{}, F32{}, four) : run(E{}, F32{}, one);
        return dim >= 8 ? run(E{}, E{}, eight) : run(E{}, E{}, one);
    };
    return dtype == SPMV_F16 ? half(F16{}) : half(BF16{});
}

extern "C" spmv_status embed_grad_workspace_size(int32_t n_tok, int32_t n_vocab, int32_t dim, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_table(n_tok, n_vocab, dim, SPMV_F32);
    if (st != SPMV_OK) return st;
    if (n_tok > ER_MAX_TOK) return fail(SPMV_ERR_UNSUPPORTED, "more than %d tokens are not supported", ER_MAX_TOK);
    *bytes = parts_of(n_tok, dim).total;
    return SPMV_OK;
}

extern "C" spmv_status embed_grad(int32_t n_tok, int32_t n_vocab, int32_t dim, int32_t dtype, const int32_t *ids,
                                  const void *dy, int64_t lddy, float scale, int32_t accumulate, float *dtable,
                                  int64_t lddt, void *workspace, size_t workspace_bytes, void *stream) {
    spmv_status st = check_table(n_tok, n_vocab, dim, dtype);
    if (st != SPMV_OK) return st;
    size_t need = 0;
    st = embed_grad_workspace_size(n_tok, n_vocab, dim, &need);
    if (st != SPMV_OK) return st;
    if (lddy < dim || lddt < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_vocab == 0 || dim == 0 || (n_tok == 0 && accumulate)) return SPMV_OK;
    if (!dtable || (n_tok > 0 && (!ids || !dy))) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (need && !workspace)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (embed_grad_workspace_size gives its size)");
    if (workspace_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    const bool add = accumulate != 0;
    const bool wide = dim >= 4;
    const int vec = wide ? 4 : 1;
    const int per = (int)per_block(n_tok), n_blocks = (int)ceil_div(n_tok, per), pieces = (int)ceil_div(dim, 64 * vec);
    const int64_t waves = (int64_t)n_blocks * pieces;
    st = check_grid(ceil_div(waves, 4));
    if (st != SPMV_OK) return st;
    st = check_grid(ceil_div((int64_t)n_vocab * dim, EG_CLEAR) + ceil_div(n_tok, 64), 1024);
    if (st != SPMV_OK) return st;
    if (pieces > 65535) return fail(SPMV_ERR_UNSUPPORTED, "rows of %d elements are not supported", dim);
    const Parts p = parts_of(n_tok, dim);
    char *base = static_cast<char *>(workspace);
    int *sorted = reinterpret_cast<int *>(base), *order = reinterpret_cast<int *>(base + p.ints);
    float *heads = reinterpret_cast<float *>(base + p.ints * (p.digits ? 4 : 2) + p.counts);
    hipStream_t s = as_stream(stream);
    const int sort_blocks = p.digits ? p.chunks : (int)ceil_div(n_tok, 64);
    Fill fill = {dtable, lddt, n_vocab, dim, sort_blocks, 0};
    if (!add) fill.blocks = (int)ceil_div((int64_t)n_vocab * dim, EG_CLEAR);
    if (p.digits) {
        int *other = reinterpret_cast<int *>(base + 2 * p.ints), *other_order = reinterpret_cast<int *>(base + 3 * p.ints);
        int *counts = reinterpret_cast<int *>(base + 4 * p.ints);
        int bits = 1;
        while (bits < 31 && (n_vocab >> bits) != 0) ++bits;          // keys 0 .. n_vocab
        const int passes = (bits + ER_BITS - 1) / ER_BITS;
        for (int i = 0; i < passes; ++i) {
            // the last pass ends in sorted and order
            const bool to = (passes - 1 - i) % 2 == 0;
            int *ko = to ? sorted : other, *oo = to ? order : other_order;
            const int *ki = to ? other : sorted, *oi = to ? other_order : order;
            if (i == 0) {
                k_embed_count<true><<<p.chunks + fill.blocks, 1024, 0, s>>>(n_tok, n_vocab, 0, p.chunks, ids, counts, fill);
                SPMV_LAUNCHED("k_embed_count");
            } else {
                k_embed_count<false><<<p.chunks, 1024, 0, s>>>(n_tok, n_vocab, ER_BITS * i, p.chunks, ki, counts, fill);
                SPMV_LAUNCHED("k_embed_count");
            }
            k_embed_scan<<<1, 1024, 0, s>>>(p.chunks * ER_BINS, counts);
            SPMV_LAUNCHED("k_embed_scan");
            if (i == 0)
                k_embed_scatter<true><<<p.chunks, 1024, 0, s>>>(n_tok, n_vocab, 0, p.chunks, ids, nullptr, counts, ko, oo);
            else
                k_embed_scatter<false><<<p.chunks, 1024, 0, s>>>(n_tok, n_vocab, ER_BITS * i, p.chunks, ki, oi, counts, ko, oo);
            SPMV_LAUNCHED("k_embed_scatter");
        }
    } else {
        k_embed_rank<<<sort_blocks + fill.blocks, 1024, 0, s>>>(n_tok, n_vocab, ids, sorted, order, fill);
        SPMV_LAUNCHED("k_embed_rank");
    }
    if (waves > 0) {
        auto sum = [&](auto e, auto v) {
            typedef decltype(e) E;
            constexpr int VEC = decltype(v)::value;
            k_embed_sum<E, VEC><<<(int)ceil_div(waves, 4), 256, 0, s>>>(
                n_tok, n_vocab, dim, per, n_blocks, pieces, sorted, order, static_cast<const typename E::T *>(dy), lddy,
                scale, add, dtable, lddt, heads);
        };
        // 4 columns for a lane: 16 bytes of the table
        auto by_width = [&](auto e) {
            wide ? sum(e, std::integral_constant<int, 4>{}) : sum(e, std::integral_constant<int, 1>{});
        };
        dtype == SPMV_F32 ? by_width(F32{}) : dtype == SPMV_F16 ? by_width(F16{}) : by_width(BF16{});
        SPMV_LAUNCHED("k_embed_sum");
    }
    if (n_blocks > 1) {
        const dim3 grid(n_blocks - 1, pieces);
        if (vec == 4)
            k_embed_join<4><<<grid, 64 * EJ_WAVES, 0, s>>>(n_tok, n_vocab, dim, per, n_blocks, sorted, scale, add, dtable, lddt, heads);
        else
            k_embed_join<1><<<grid, 64 * EJ_WAVES, 0, s>>>(n_tok, n_vocab, dim, per, n_blocks, sorted, scale, add, dtable, lddt, heads);
        SPMV_LAUNCHED("k_embed_join");
    }
    return SPMV_OK;
}
