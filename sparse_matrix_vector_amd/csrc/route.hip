// Tokens sorted by group (expert or adapter) and back, on gfx950.
//
// The plan is a stable counting sort of n_slots keys, the many-token form of
// the row grouping of the CSR planner: slot s = (token s / k, choice s % k)
// carries a group key; offsets[g] counts the slots of smaller groups, order
// lists the slots group by group in ascending slot order, pos is its inverse,
// and keys outside [0, n_groups) are dropped (pos -1, last in order).  With P
// the n_slots x n_tok 0/1 matrix of that order, the gather is P x, the combine
// is (P^T diag) ys, an ELL product with k slots per token, and each is the
// other's gradient.
//
// All three data kernels stream their rows once with 16-byte accesses and are
// bound by HBM; sums run in fp32 over ascending choices, so results do not
// depend on scheduling.
#include "elem.hpp"

#include <algorithm>
#include <type_traits>

namespace spmv {
namespace {

constexpr int RT_TILE = 16;          // rows of a plan tile
constexpr int RT_MAX_GROUPS = 2048;  // bins of the sort in LDS (limit of the 4-wave form)
constexpr int RT_WIDE_BINS = 896;    // above: 4 waves per workgroup, so that a counter per wave and bin fits 64 KB
constexpr int RT_MAX_SLOTS = 1 << 22; // every workgroup sums the counts of all chunks
constexpr int RT_CHUNK = 4096;       // slots per workgroup of the 16-wave form (256 per wave), 1024 of the 4-wave form

// Up to RT_ONE slots are sorted by one workgroup in one launch; more are counted
// per chunk first.  64 groups: 6000 slots 8.7 us in one launch, 9.5 counted first;
// 8192 slots 10.6 and 9.7, which the second launch costs the host three times over.
constexpr int RT_ONE = 8192;

inline int sort_waves(int n_groups) { return n_groups + 1 <= RT_WIDE_BINS ? 16 : 4; }
inline int64_t sort_blocks(int64_t n_slots, int n_groups) {
    const int waves = sort_waves(n_groups);
    return n_slots <= RT_ONE ? 1 : ceil_div(n_slots, waves * (RT_CHUNK / 16));
}

__device__ __forceinline__ int bin_of(int key, int n_groups) {
    return (unsigned)key < (unsigned)n_groups ? key : n_groups;
}

// Slots per bin of each chunk of the keys (several workgroups): 4.7 us for 65528
// slots, and 7.7 us for the sort after it; both are short chains of LDS steps.
__global__ __launch_bounds__(1024) void k_route_count(int n_slots, int n_groups, int chunk,
                                                      const int *__restrict__ keys, int *__restrict__ counts) {
    extern __shared__ int hist[];
    const int nb = n_groups + 1;
    for (int g = threadIdx.x; g < nb; g += blockDim.x) hist[g] = 0;
    __syncthreads();
    const int s0 = blockIdx.x * chunk, s1 = min(n_slots, s0 + chunk);
    for (int s = s0 + threadIdx.x; s < s1; s += blockDim.x) atomicAdd(&hist[bin_of(keys[s], n_groups)], 1);
    __syncthreads();
    for (int g = threadIdx.x; g < nb; g += blockDim.x) counts[(size_t)blockIdx.x * nb + g] = hist[g];
}

// Sorts chunk blockIdx.x of the keys.  LDS: a counter per wave and bin, then
// the first position and the first tile of every bin.  A wave's slots are
// consecutive, so (chunk, wave, step, lane) is slot order and the sort is
// stable: equal keys of one step are ranked by ballots over the key's bits.
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_route_sort(int n_slots, int n_groups, int key_bits, int per_wave,
                                                           const int *__restrict__ keys,
                                                           const int *__restrict__ counts,
                                                           int *__restrict__ offsets, int *__restrict__ order,
                                                           int *__restrict__ pos, int4 *__restrict__ tiles,
                                                           int n_tiles) {
    extern __shared__ int lds[];
    const int nb = n_groups + 1;
    int *off = lds + WAVES * nb;       // nb + 1
    int *toff = off + nb + 1;          // nb + 1
    const int lane = __lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int *mine = lds + wv * nb;
    const int chunk = per_wave * WAVES;
    const int s0 = min((int64_t)n_slots, (int64_t)blockIdx.x * chunk + (int64_t)wv * per_wave);
    const int s1 = min(n_slots, s0 + per_wave);

    for (int i = threadIdx.x; i < WAVES * nb + 2 * (nb + 1); i += 64 * WAVES) lds[i] = 0;
    __syncthreads();
    for (int s = s0 + lane; s < s1; s += 64) atomicAdd(&mine[bin_of(keys[s], n_groups)], 1);
    // slots per bin over all chunks (toff) and over the chunks before this one (off)
    if (gridDim.x > 1) {
        const int n = gridDim.x * nb;
        for (int i = threadIdx.x; i < n; i += 64 * WAVES) {
            const int b = i / nb, g = i - b * nb, c = counts[i];
            if (c) {
                atomicAdd(&toff[g], c);
                if (b < (int)blockIdx.x) atomicAdd(&off[g], c);
            }
        }
    }
    __syncthreads();
    for (int g = threadIdx.x; g < nb; g += 64 * WAVES) {
        int run = off[g];
        for (int w = 0; w < WAVES; ++w) {
            const int c = lds[w * nb + g];
            lds[w * nb + g] = run;
            run += c;
        }
        if (gridDim.x == 1) toff[g] = run;
    }
    __syncthreads();
    // exclusive scans of the bin sizes and of their tiles
    if (wv == 0) {
        int base = 0, tbase = 0;
        for (int g0 = 0; g0 <= nb; g0 += 64) {
            const int g = g0 + lane;
            const int c = g < nb ? toff[g] : 0;
            const int t = (c + RT_TILE - 1) / RT_TILE;
            const int ci = wave_inclusive_scan(c), ti = wave_inclusive_scan(t);
            if (g <= nb) {
                off[g] = base + ci - c;
                toff[g] = tbase + ti - t;
            }
            base += __builtin_amdgcn_readlane(ci, 63);
            tbase += __builtin_amdgcn_readlane(ti, 63);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int g = threadIdx.x; g <= n_groups; g += 64 * WAVES) offsets[g] = off[g];
    for (int t = blockIdx.x * 64 * WAVES + threadIdx.x; t < n_tiles; t += gridDim.x * 64 * WAVES) {
        int4 e = make_int4(-1, 0, 0, 0);
        if (t < toff[nb]) {
            int lo = 0, hi = nb - 1;              // the last bin whose first tile is <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (toff[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int b = off[lo] + (t - toff[lo]) * RT_TILE;
            e = make_int4(lo < n_groups ? lo : -1, b, min(b + RT_TILE, off[lo + 1]), off[lo]);
        }
        tiles[t] = e;
    }
    for (int s = s0; s < s1; s += 64) {           // uniform: every lane takes part in the ballots
        const bool in = s + lane < s1;
        const int g = in ? bin_of(keys[s + lane], n_groups) : 0;
        unsigned long long same = __ballot(in);
        for (int b = 0; b < key_bits; ++b) {
            const unsigned long long ones = __ballot((g >> b) & 1);
            same &= ((g >> b) & 1) ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int lead = in ? __ffsll(same) - 1 : lane;
        int at = 0;
        if (in && lane == lead) at = atomicAdd(&mine[g], __popcll(same));
        at = __shfl(at, lead);
        if (in) {
            const int p = off[g] + at + rank;
            order[p] = s + lane;
            pos[s + lane] = g < n_groups ? p : -1;
        }
    }
}

// Row pieces: a wave moves COLS elements of one row, VEC per lane and access.
// Rows are moved 16 bytes at a time whatever their alignment; the last access
// of a row whose width is not a multiple of VEC starts early and overlaps the
// one before it.
template <typename E, int VEC>
constexpr int piece_accesses() { return VEC > 1 ? 4 : 8; }

// xs[pos[t, c]] = w[t, c] * x[t]: a wave reads a piece of a token's row once and
// writes it to every choice's place: 54 us for 8191 tokens of 2048 bf16 with
// k = 8 (302 MB, 5.6 TB/s).  By sorted rows, each x row read k times, 73 us.
template <typename E, int VEC>
__global__ __launch_bounds__(256) void k_route_gather(int n_tok, int n_slots, int k, int dim, int pieces,
                                                      const int *__restrict__ pos, const float *__restrict__ w,
                                                      const typename E::T *__restrict__ x, int64_t ldx,
                                                      typename E::T *__restrict__ xs, int64_t ldxs) {
    typedef typename E::T T;
    constexpr int U = piece_accesses<E, VEC>(), COLS = 64 * VEC * U;
    const int lane = __lane_id();
    const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tok = (int)(id / pieces), piece = (int)(id - (int64_t)tok * pieces);
    if (tok >= n_tok) return;
    const T *src = x + (int64_t)tok * ldx;
    const int c0 = piece * COLS + lane * VEC;
    Vec<E, VEC> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_any<E, VEC>(src + min(c0 + u * 64 * VEC, dim - VEC));
    for (int j = 0; j < k; ++j) {
        const int64_t s = (int64_t)tok * k + j;
        const int p = pos[s];
        if ((unsigned)p >= (unsigned)n_slots) continue;
        const float f = w ? w[s] : 1.0f;
        T *dst = xs + (int64_t)p * ldxs;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 64 * VEC;
            if (c < dim) {
                Vec<E, VEC> o = v[u];
                if (w) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o.v[i] = (T)(f * (float)v[u].v[i]);
                }
                store_once<E, VEC>(dst + min(c, dim - VEC), o);
            }
        }
    }
}

// y[t] = sum over choices c (ascending) of w[t, c] * ys[pos[t, c]], rounded once:
// 54 us at the same sizes (302 MB, 5.6 TB/s).
template <typename E, int VEC>
__global__ __launch_bounds__(256) void k_route_combine(int n_tok, int n_slots, int k, int dim, int pieces,
                                                       const int *__restrict__ pos, const float *__restrict__ w,
                                                       const typename E::T *__restrict__ ys, int64_t ldys,
                                                       typename E::T *__restrict__ y, int64_t ldy) {
    typedef typename E::T T;
    // fewer columns per wave than the gather: the loads of 8 choices' rows are in flight together
    constexpr int U = VEC > 1 ? 1 : 4, COLS = 64 * VEC * U, KU = VEC > 1 ? 8 : 4;
    const int lane = __lane_id();
    const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tok = (int)(id / pieces), piece = (int)(id - (int64_t)tok * pieces);
    if (tok >= n_tok) return;
    const int c0 = piece * COLS + lane * VEC;
    float acc[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[u][i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KU) {
        Vec<E, VEC> v[KU][U];
        float f[KU];
        int p[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const int64_t s = (int64_t)tok * k + min(j0 + j, k - 1);
            p[j] = j0 + j < k ? pos[s] : -1;
            f[j] = w ? w[s] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < KU; ++j)
            if ((unsigned)p[j] < (unsigned)n_slots) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    v[j][u] = load_once<E, VEC>(ys + (int64_t)p[j] * ldys + min(c0 + u * 64 * VEC, dim - VEC));
            }
#pragma unroll
        for (int j = 0; j < KU; ++j)
            if ((unsigned)p[j] < (unsigned)n_slots) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[u][i] = fmaf(f[j], (float)v[j][u].v[i], acc[u][i]);
            }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * VEC;
        if (c < dim) {
            Vec<E, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.v[i] = (T)acc[u][i];
            store_any<E, VEC>(y + (int64_t)tok * ldy + min(c, dim - VEC), o);
        }
    }
}

// dys[pos[t, c]] = w[t, c] * dy[t] and dw[t, c] = <ys[pos[t, c]], dy[t]>: one
// workgroup per token, so each row of dy is read once per 8 choices: 106 us at
// the same sizes (570 MB, 5.4 TB/s).
template <typename E, int VEC>
__global__ __launch_bounds__(256) void k_route_combine_grad(int n_slots, int k, int dim,
                                                            const typename E::T *__restrict__ dy, int64_t lddy,
                                                            const typename E::T *__restrict__ ys, int64_t ldys,
                                                            const int *__restrict__ pos,
                                                            const float *__restrict__ w,
                                                            typename E::T *__restrict__ dys, int64_t lddys,
                                                            float *__restrict__ dw) {
    typedef typename E::T T;
    constexpr int KU = 8;
    __shared__ float part[4][KU];
    const int lane = __lane_id(), wv = threadIdx.x / 64;
    const int tok = blockIdx.x;
    const T *dyr = dy + (int64_t)tok * lddy;
    for (int j0 = 0; j0 < k; j0 += KU) {
        int p[KU];
        float f[KU], acc[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const int64_t s = (int64_t)tok * k + min(j0 + j, k - 1);
            p[j] = j0 + j < k ? pos[s] : -1;
            f[j] = w ? w[s] : 1.0f;
            acc[j] = 0.0f;
        }
        for (int c = threadIdx.x * VEC; c < dim; c += 256 * VEC) {
            const int at = min(c, dim - VEC);
            const Vec<E, VEC> g = load_any<E, VEC>(dyr + at);
            Vec<E, VEC> v[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if ((unsigned)p[j] < (unsigned)n_slots) v[j] = load_once<E, VEC>(ys + (int64_t)p[j] * ldys + at);
            // what the access before has already counted is left out of the sum
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if ((unsigned)p[j] < (unsigned)n_slots) {
                    Vec<E, VEC> o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        acc[j] = at + i >= c ? fmaf((float)v[j].v[i], (float)g.v[i], acc[j]) : acc[j];
                        o.v[i] = (T)(f[j] * (float)g.v[i]);
                    }
                    store_once<E, VEC>(dys + (int64_t)p[j] * lddys + at, o);
                }
        }
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const float s = wave_sum(acc[j]);
            if (lane == 0) part[wv][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < KU && j0 + (int)threadIdx.x < k)
            dw[(int64_t)tok * k + j0 + threadIdx.x] =
                (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
spmv_status check_plan_shape(int64_t n_slots, int64_t n_groups) {
    if (n_slots < 0 || n_groups < 1) return fail(SPMV_ERR_INVALID_VALUE, "n_slots must be >= 0 and n_groups >= 1");
    if (n_groups > RT_MAX_GROUPS)
        return fail(SPMV_ERR_UNSUPPORTED, "more than %d groups are not supported", RT_MAX_GROUPS);
    if (n_slots > RT_MAX_SLOTS) return fail(SPMV_ERR_UNSUPPORTED, "more than %d slots are not supported", RT_MAX_SLOTS);
    return SPMV_OK;
}

int64_t tile_count(int64_t n_slots, int64_t n_groups) {
    return (n_slots + (RT_TILE - 1) * std::min(n_groups + 1, n_slots)) / RT_TILE;
}

spmv_status check_rows(int32_t n_tok, int32_t top_k, int32_t dim, int32_t dtype) {
    if (n_tok < 0 || dim < 0 || top_k < 1) return fail(SPMV_ERR_INVALID_VALUE, "negative size or top_k < 1");
    if (!dtype_ok(dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", dtype);
    if ((int64_t)n_tok * top_k > INT32_MAX) return fail(SPMV_ERR_OVERFLOW, "n_tok * top_k does not fit int32");
    return SPMV_OK;
}

// whether a row holds at least one 16-byte access
bool wide_rows(int32_t dim, int32_t dtype) { return (size_t)dim * dtype_size(dtype) >= 16; }

template <typename F>
spmv_status by_type(int32_t dtype, bool vec, F f) {
    if (dtype == SPMV_F16) return vec ? f(F16{}, std::integral_constant<int, 8>{}) : f(F16{}, std::integral_constant<int, 1>{});
    if (dtype == SPMV_BF16) return vec ? f(BF16{}, std::integral_constant<int, 8>{}) : f(BF16{}, std::integral_constant<int, 1>{});
    return vec ? f(F32{}, std::integral_constant<int, 4>{}) : f(F32{}, std::integral_constant<int, 1>{});
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status route_tile_count(int32_t n_slots, int32_t n_groups, int32_t *n_tiles) {
    if (!n_tiles) return fail(SPMV_ERR_INVALID_VALUE, "n_tiles is NULL");
    const spmv_status st = check_plan_shape(n_slots, n_groups);
    if (st != SPMV_OK) return st;
    *n_tiles = (int32_t)tile_count(n_slots, n_groups);
    return SPMV_OK;
}

extern "C" spmv_status route_workspace_size(int32_t n_slots, int32_t n_groups, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_plan_shape(n_slots, n_groups);
    if (st != SPMV_OK) return st;
    const int64_t nb = sort_blocks(n_slots, n_groups);
    *bytes = nb == 1 ? 0 : ((size_t)nb * (size_t)(n_groups + 1) * 4 + 255) & ~size_t(255);
    return SPMV_OK;
}

extern "C" spmv_status route_plan(int32_t n_slots, int32_t n_groups, const int32_t *keys, int32_t *offsets,
                                  int32_t *order, int32_t *pos, int32_t *tiles, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    spmv_status st = check_plan_shape(n_slots, n_groups);
    if (st != SPMV_OK) return st;
    if (!offsets || (n_slots > 0 && (!keys || !order || !pos || !tiles)))
        return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (!aligned16(tiles)) return fail(SPMV_ERR_UNSUPPORTED, "tiles must be 16-byte aligned");
    size_t need = 0;
    route_workspace_size(n_slots, n_groups, &need);
    if (need && !workspace) return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (route_workspace_size gives its size)");
    if (need > workspace_bytes)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 3u) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 4-byte aligned");
    hipStream_t s = as_stream(stream);
    const int nb = (int)sort_blocks(n_slots, n_groups);
    const int waves = sort_waves(n_groups);
    int *counts = static_cast<int *>(workspace);
    int bits = 0;
    while ((n_groups >> bits) != 0) ++bits;              // keys 0 .. n_groups
    const int n_tiles = (int)tile_count(n_slots, n_groups);
    const int chunk = waves * (RT_CHUNK / 16);
    const int per_wave = nb == 1 ? (int)(ceil_div(std::max(n_slots, 1), waves * 64) * 64) : RT_CHUNK / 16;
    const size_t lds = ((size_t)waves * (n_groups + 1) + 2 * (size_t)(n_groups + 2)) * sizeof(int);
    if (nb > 1) {
        k_route_count<<<nb, 64 * waves, (size_t)(n_groups + 1) * sizeof(int), s>>>(n_slots, n_groups, chunk, keys, counts);
        SPMV_LAUNCHED("k_route_count");
    }
    if (waves == 16)
        k_route_sort<16><<<nb, 1024, lds, s>>>(n_slots, n_groups, bits, per_wave, keys, counts, offsets, order, pos,
                                               reinterpret_cast<int4 *>(tiles), n_tiles);
    else
        k_route_sort<4><<<nb, 256, lds, s>>>(n_slots, n_groups, bits, per_wave, keys, counts, offsets, order, pos,
                                             reinterpret_cast<int4 *>(tiles), n_tiles);
    SPMV_LAUNCHED("k_route_sort");
    return SPMV_OK;
}

extern "C" spmv_status route_gather(int32_t n_tok, int32_t top_k, int32_t dim, int32_t dtype, const int32_t *pos,
                                    const float *weights, const void *x, int64_t ldx, void *xs, int64_t ldxs,
                                    void *stream) {
    spmv_status st = check_rows(n_tok, top_k, dim, dtype);
    if (st != SPMV_OK) return st;
    if (ldx < dim || ldxs < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_tok == 0 || dim == 0) return SPMV_OK;
    if (!pos || !x || !xs) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    const int n_slots = n_tok * top_k;
    return by_type(dtype, wide_rows(dim, dtype), [&](auto e, auto vec) {
        typedef decltype(e) E;
        constexpr int VEC = decltype(vec)::value;
        const int pieces = (int)ceil_div(dim, 64 * VEC * piece_accesses<E, VEC>());
        const int64_t blocks = ceil_div((int64_t)n_tok * pieces, 4);
        const spmv_status s = check_grid(blocks);
        if (s != SPMV_OK) return s;
        k_route_gather<E, VEC><<<(int)blocks, 256, 0, as_stream(stream)>>>(
            n_tok, n_slots, top_k, dim, pieces, pos, weights, static_cast<const typename E::T *>(x), ldx,
            static_cast<typename E::T *>(xs), ldxs);
        SPMV_LAUNCHED("k_route_gather");
        return SPMV_OK;
    });
}

extern "C" spmv_status route_combine(int32_t n_tok, int32_t top_k, int32_t dim, int32_t dtype, const int32_t *pos,
                                     const float *weights, const void *ys, int64_t ldys, void *y, int64_t ldy,
                                     void *stream) {
    spmv_status st = check_rows(n_tok, top_k, dim, dtype);
    if (st != SPMV_OK) return st;
    if (ldys < dim || ldy < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_tok == 0 || dim == 0) return SPMV_OK;
    if (!pos || !ys || !y) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    const int n_slots = n_tok * top_k;
    return by_type(dtype, wide_rows(dim, dtype), [&](auto e, auto vec) {
        typedef decltype(e) E;
        constexpr int VEC = decltype(vec)::value;
        const int pieces = (int)ceil_div(dim, 64 * VEC * (VEC > 1 ? 1 : 4));
        const int64_t blocks = ceil_div((int64_t)n_tok * pieces, 4);
        const spmv_status s = check_grid(blocks);
        if (s != SPMV_OK) return s;
        k_route_combine<E, VEC><<<(int)blocks, 256, 0, as_stream(stream)>>>(
            n_tok, n_slots, top_k, dim, pieces, pos, weights, static_cast<const typename E::T *>(ys), ldys,
            static_cast<typename E::T *>(y), ldy);
        SPMV_LAUNCHED("k_route_combine");
        return SPMV_OK;
    });
}

extern "C" spmv_status route_combine_grad(int32_t n_tok, int32_t top_k, int32_t dim, int32_t dtype, const void *dy,
                                          int64_t lddy, const void *ys, int64_t ldys, const int32_t *pos,
                                          const float *weights, void *dys, int64_t lddys, float *dw, void *stream) {
    spmv_status st = check_rows(n_tok, top_k, dim, dtype);
    if (st != SPMV_OK) return st;
    if (lddy < dim || ldys < dim || lddys < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_tok == 0) return SPMV_OK;
    if (!pos || !dw || (dim > 0 && (!dy || !ys || !dys))) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    st = check_grid(n_tok);
    if (st != SPMV_OK) return st;
    return by_type(dtype, wide_rows(dim, dtype), [&](auto e, auto vec) {
        typedef decltype(e) E;
        typedef typename E::T T;
        constexpr int VEC = decltype(vec)::value;
        k_route_combine_grad<E, VEC><<<n_tok, 256, 0, as_stream(stream)>>>(
            n_tok * top_k, top_k, dim, static_cast<const T *>(dy), lddy, static_cast<const T *>(ys), ldys, pos, weights,
            static_cast<T *>(dys), lddys, dw);
        SPMV_LAUNCHED("k_route_combine_grad");
        return SPMV_OK;
    });
}
