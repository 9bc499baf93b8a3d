// Low-rank adapters of many requests beside a shared projection, on gfx950.
//
// Token t with adapter a adds  scale[a] * B[a]^T (A[a] x_t)  to its row of the
// projection's output.  A [n, r, n_in] and B [n, r, n_out] are both rank-major,
// so the gradient in x is the same product with A and B exchanged, and the
// weight gradients are two sums of outer products over an adapter's tokens:
//   dA[a][j, :] = scale * sum_t (B[a] dy_t)_j x_t,   dB[a][j, :] = scale * sum_t (A[a] x_t)_j dy_t.
//
// Tokens come grouped by adapter (a route plan of one choice per token); a
// tile is up to 16 tokens of one adapter, the M of a 16x16x32 matrix
// instruction.  Three kernels:
//   shrink  h = A x: contraction over the long axis, split over waves and
//           workgroups; each workgroup stores its own partial sum in fp32,
//           and whoever reads h adds the partials in order (no atomics, the
//           same bits on every call);
//   expand  y = y_in + scale * B^T h: the contraction is the rank.  B is read
//           16 bytes along its rows, eight rows per lane, and one v_perm per
//           row pair turns them into the operands of eight instructions, each
//           of which owns every eighth column; a lane then holds eight
//           neighbouring columns of the result;
//   outer   dA or dB: the contraction is the tokens, x (dy) is read the same
//           way as B.
// h stays fp32 in memory.  As an operand it is split into a sum of two 16-bit
// numbers (fp16, after scaling by a power of two so that neither part
// overflows or vanishes: 22 bits) or three (bf16 with an fp32 result: 24 bits;
// two, 16 bits, when the result is rounded to bf16 anyway), so the rank
// vector loses nothing that the result could show.
#include "elem.hpp"

#include <algorithm>
#include <type_traits>

namespace spmv {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int LR_TILE = 16;         // tokens per plan tile
constexpr int LR_MAX_RANK = 128;
constexpr int LR_MAX_SPLIT = 32;
constexpr int LR_WAVE_COLS = 128;   // columns of a wave in expand and outer: 16 lanes x 8

template <typename E>
struct Frag;
template <>
struct Frag<F16> {
    typedef h8 V;
    static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<BF16> {
    typedef b8 V;
    static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

// Elements c .. c + 7 of a row as 16 bytes; those at or past n are zero.
// VEC: n is a multiple of 8 and the row 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const unsigned short *__restrict__ row, int c, int n) {
    if (VEC) return c < n ? *reinterpret_cast<const u32x4 *>(row + c) : u32x4{0u, 0u, 0u, 0u};
    unsigned short v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? row[c + i] : (unsigned short)0;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (unsigned int)v[2 * i] | ((unsigned int)v[2 * i + 1] << 16);
    return r;
}

// Eight rows of eight 16-bit elements (row i in r[i]) as eight operands:
// operand c holds element c of rows 0 .. 7.
__device__ __forceinline__ u32x4 column_of(const u32x4 (&r)[8], int c) {
    const unsigned int sel = (c & 1) ? 0x07060302u : 0x05040100u;   // high or low halves of {row i + 1, row i}
    u32x4 o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = __builtin_amdgcn_perm(r[2 * p + 1][c >> 1], r[2 * p][c >> 1], sel);
    return o;
}

struct ShrinkArg {
    const unsigned short *x, *W;   // x [n_tok, dim] with row stride ldx; W [n_adapters, max_rank, dim]
    int64_t ldx;
    int dim;
    float *h;                      // [split][n_tok][16 NJ], rows in sorted order
};

__device__ __forceinline__ int rank_of(const int *ranks, int a, int max_rank) {
    return ranks ? min(max(ranks[a], 0), max_rank) : max_rank;
}

// One workgroup: tile blockIdx.x, k range blockIdx.y of gridDim.y, product
// blockIdx.z (the gradient needs A x and B dy).  Each of the 4 waves takes a
// quarter of the range in steps of 64 (lane group q owns k = 16 q .. 16 q + 15
// of a step, in x and W alike), and wave 0 adds the four sums.
template <typename E, int NJ, bool VEC>
__global__ __launch_bounds__(256) void k_lora_shrink(int n_tok, int n_adapters, int max_rank,
                                                     const int *__restrict__ ranks,
                                                     const int *__restrict__ order,
                                                     const int4 *__restrict__ tiles, ShrinkArg a0, ShrinkArg a1) {
    typedef typename Frag<E>::V V;
    __shared__ f32x4 part[3][NJ][64];
    const ShrinkArg &a = blockIdx.z ? a1 : a0;
    const int4 tile = tiles[blockIdx.x];
    if ((unsigned)tile.x >= (unsigned)n_adapters) return;
    const int rank = rank_of(ranks, tile.x, max_rank);
    const int nj = (rank + 15) / 16;
    if (nj == 0) return;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tok = order[min(tile.y + n, tile.z - 1)];
    const unsigned short *xr = a.x + (int64_t)tok * a.ldx;
    const unsigned short *wr[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        wr[j] = a.W + ((int64_t)tile.x * max_rank + min(16 * j + n, max_rank - 1)) * a.dim;
    // steps of this wave: waves of all splits take turns over 64-wide steps in contiguous runs
    const int steps = (a.dim + 63) / 64, parts = gridDim.y * 4, mine = blockIdx.y * 4 + wv;
    const int lo = (int)((int64_t)steps * mine / parts), hi = (int)((int64_t)steps * (mine + 1) / parts);
    f32x4 acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = lo; s < hi; ++s) {
        const int k = s * 64 + q * 16;
        const u32x4 x0 = load8<VEC>(xr, k, a.dim), x1 = load8<VEC>(xr, k + 8, a.dim);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if (j < nj) {
                const u32x4 w0 = load8<VEC>(wr[j], k, a.dim), w1 = load8<VEC>(wr[j], k + 8, a.dim);
                acc[j] = Frag<E>::mma(__builtin_bit_cast(V, x0), __builtin_bit_cast(V, w0), acc[j]);
                acc[j] = Frag<E>::mma(__builtin_bit_cast(V, x1), __builtin_bit_cast(V, w1), acc[j]);
            }
        }
    }
    if (wv > 0) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) part[wv - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wv > 0) return;
    float *h = a.h + (int64_t)blockIdx.y * n_tok * (16 * NJ);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const f32x4 v = (acc[j] + part[0][j][lane]) + (part[1][j][lane] + part[2][j][lane]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = tile.y + 4 * q + i;     // D: row 4 q + i, column n
            if (row < tile.z) h[(int64_t)row * (16 * NJ) + 16 * j + n] = 16 * j + n < rank ? v[i] : 0.0f;
        }
    }
}

// v as a sum of NT numbers of type E.
template <typename E, int NT>
__device__ __forceinline__ void split_terms(float v, unsigned short (&t)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const typename E::T p = (typename E::T)v;
        t[i] = __builtin_bit_cast(unsigned short, p);
        v -= (float)p;
    }
}

// The power of two that brings max |v| = m into [1, 2) (1 for 0, infinities and NaN).
__device__ __forceinline__ int scale_exponent(float m) {
    const int e = (__float_as_int(m) >> 23) & 255;
    return e == 0 || e == 255 ? 0 : 127 - e;
}

// Eight neighbouring results of one token.
template <typename Y, bool VEC>
__device__ __forceinline__ void load_row8(const typename Y::T *p, int c, int n, float (&v)[8]) {
    if (VEC) {
        constexpr int PER = 16 / (int)sizeof(typename Y::T);
#pragma unroll
        for (int i = 0; i < 8; i += PER) {
            const Vec<Y, PER> r = load_vec<Y, PER>(p + c + i);
#pragma unroll
            for (int k = 0; k < PER; ++k) v[i + k] = (float)r.v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? (float)p[c + i] : 0.0f;
    }
}
template <typename Y, bool VEC>
__device__ __forceinline__ void store_row8(typename Y::T *p, int c, int n, const float (&v)[8]) {
    if (VEC) {
        constexpr int PER = 16 / (int)sizeof(typename Y::T);
#pragma unroll
        for (int i = 0; i < 8; i += PER) {
            Vec<Y, PER> r;
#pragma unroll
            for (int k = 0; k < PER; ++k) r.v[k] = (typename Y::T)v[i + k];
            store_vec<Y, PER>(p + c + i, r);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) p[c + i] = (typename Y::T)v[i];
    }
}

// One workgroup: tile blockIdx.x, columns 512 blockIdx.y ..; 128 per wave.
template <typename E, typename Y, int NJ, int NT, bool VEC>
__global__ __launch_bounds__(256) void k_lora_expand(int n_tok, int n_adapters, int max_rank, int split,
                                                     const int *__restrict__ ranks,
                                                     const float *__restrict__ scale,
                                                     const int *__restrict__ order,
                                                     const int4 *__restrict__ tiles, const float *__restrict__ h,
                                                     const unsigned short *__restrict__ B, int dim,
                                                     const typename Y::T *y_in, int64_t ldyin,
                                                     typename Y::T *y, int64_t ldy) {
    typedef typename Frag<E>::V V;
    constexpr int R = 16 * NJ, LD = R + 8;
    __shared__ __attribute__((aligned(16))) unsigned short hs[NT][LR_TILE][LD];
    __shared__ float unscale[LR_TILE];
    const int4 tile = tiles[blockIdx.x];
    if (tile.y >= tile.z) return;
    const bool adapted = (unsigned)tile.x < (unsigned)n_adapters;
    const int rank = adapted ? rank_of(ranks, tile.x, max_rank) : 0;
    if (rank == 0 && y_in == y) return;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int c0 = blockIdx.y * (4 * LR_WAVE_COLS) + wv * LR_WAVE_COLS + 8 * n;

    if (rank > 0) {
        // 16 lanes per token: the partial sums of h in order, the token's
        // largest |h|, and the scaled terms
        const int t = threadIdx.x >> 4, l = threadIdx.x & 15;
        const int64_t row = min(tile.y + t, tile.z - 1);
        float v[NJ], m = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) v[j] = 0.0f;
        for (int s = 0; s < split; ++s)
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] += h[((int64_t)s * n_tok + row) * R + 16 * j + l];
#pragma unroll
        for (int j = 0; j < NJ; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
        for (int d = 1; d < 16; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
        const int e = E::CODE == SPMV_F16 ? scale_exponent(m) : 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            unsigned short terms[NT];
            split_terms<E, NT>(ldexpf(v[j], e), terms);
#pragma unroll
            for (int i = 0; i < NT; ++i) hs[i][t][16 * j + l] = terms[i];
        }
        if (l == 0) unscale[t] = ldexpf(scale ? scale[tile.x] : 1.0f, -e);
        __syncthreads();
    }
    f32x4 acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (rank > 0) {
        const unsigned short *Br = B + (int64_t)tile.x * max_rank * dim;
        if constexpr (NJ == 1) {
            // up to 16 ranks: the terms share the contraction, eight ranks
            // of one term per lane group and step
            constexpr int STEPS = (2 * NT + 3) / 4;
            u32x4 r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = load8<VEC>(Br + (int64_t)min(8 * (q & 1) + i, max_rank - 1) * dim, c0, dim);
            const int live = rank - 8 * (q & 1);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= live) r[i] = u32x4{0u, 0u, 0u, 0u};   // rows past the rank may hold anything
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int term = 2 * s + (q >> 1);
                u32x4 a = u32x4{0u, 0u, 0u, 0u};
                if (term < NT) a = *reinterpret_cast<const u32x4 *>(&hs[term < NT ? term : 0][n][8 * (q & 1)]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    acc[c] = Frag<E>::mma(__builtin_bit_cast(V, a), __builtin_bit_cast(V, column_of(r, c)), acc[c]);
            }
        } else {
            for (int j0 = 0; j0 < rank; j0 += 32) {
                const int jb = j0 + 8 * q;
                u32x4 r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = load8<VEC>(Br + (int64_t)min(jb + i, max_rank - 1) * dim, c0, dim);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (jb + i >= rank) r[i] = u32x4{0u, 0u, 0u, 0u};
                V a[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    a[i] = __builtin_bit_cast(V, *reinterpret_cast<const u32x4 *>(&hs[i][n][jb]));
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const V b = __builtin_bit_cast(V, column_of(r, c));
#pragma unroll
                    for (int i = 0; i < NT; ++i) acc[c] = Frag<E>::mma(a[i], b, acc[c]);
                }
            }
        }
    }
    if (c0 >= dim) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = tile.y + 4 * q + i;
        if (row >= tile.z) break;
        const int64_t tok = order[row];
        float v[8];
        if (y_in)
            load_row8<Y, VEC>(y_in + tok * ldyin, c0, dim, v);
        else
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = 0.0f;
        const float f = rank > 0 ? unscale[4 * q + i] : 0.0f;
        if (rank > 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = fmaf(f, acc[c][i], v[c]);
        }
        store_row8<Y, VEC>(y + tok * ldy, c0, dim, v);
    }
}

struct OuterArg {
    const unsigned short *x;   // x or dy
    int64_t ldx;
    int dim, blocks;           // columns, and their 128-column blocks
    const float *h;            // [split][n_tok][16 NJ]
    float *out;                // [n_adapters, max_rank, dim]
};

// One workgroup: 128 columns of adapter blockIdx.y's gradient; blockIdx.x
// counts the column blocks of the first product, then of the second, and
// blockIdx.z blocks of NJ rank tiles out of the R / 16 of h.  The 8 waves take
// turns over 32-token steps and their sums are added in order.
template <typename E, int NJ, int R, int NT, bool VEC>
__global__ __launch_bounds__(512) void k_lora_outer(int n_tok, int max_rank, int split,
                                                    const int *__restrict__ ranks,
                                                    const float *__restrict__ scale,
                                                    const int *__restrict__ order,
                                                    const int *__restrict__ offsets, OuterArg a0, OuterArg a1) {
    typedef typename Frag<E>::V V;
    __shared__ f32x4 sum[8][64];
    const int r0 = blockIdx.z * 16 * NJ;   // first rank of this workgroup
    const bool second = (int)blockIdx.x >= a0.blocks;
    const OuterArg &a = second ? a1 : a0;
    const int ad = blockIdx.y;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int c0 = (blockIdx.x - (second ? a0.blocks : 0)) * LR_WAVE_COLS + 8 * n;
    const int rank = rank_of(ranks, ad, max_rank);
    const int t0 = min(max(offsets[ad], 0), n_tok), t1 = min(max(offsets[ad + 1], t0), n_tok);
    f32x4 acc[NJ][8];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int t = t0 + 32 * wv; t < t1; t += 32 * 8) {
        u32x4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t tok = order[min(t + 8 * q + i, t1 - 1)];
            r[i] = load8<VEC>(a.x + tok * a.ldx, c0, a.dim);
        }
        float g[NJ][8], m = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = min(t + 8 * q + i, t1 - 1);
                float v = 0.0f;
                for (int s = 0; s < split; ++s) v += a.h[((int64_t)s * n_tok + row) * R + r0 + 16 * j + n];
                g[j][i] = t + 8 * q + i < t1 && r0 + 16 * j + n < rank ? v : 0.0f;
                m = fmaxf(m, fabsf(g[j][i]));
            }
        int e = 0;
        if (E::CODE == SPMV_F16) {
#pragma unroll
            for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
            e = scale_exponent(m);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            u32x4 op[NT];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                unsigned short lo[NT], hi[NT];
                split_terms<E, NT>(E::CODE == SPMV_F16 ? ldexpf(g[j][i], e) : g[j][i], lo);
                split_terms<E, NT>(E::CODE == SPMV_F16 ? ldexpf(g[j][i + 1], e) : g[j][i + 1], hi);
#pragma unroll
                for (int k = 0; k < NT; ++k) op[k][i / 2] = (unsigned int)lo[k] | ((unsigned int)hi[k] << 16);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const V b = __builtin_bit_cast(V, column_of(r, c));
                f32x4 d = E::CODE == SPMV_F16 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[j][c];
#pragma unroll
                for (int k = 0; k < NT; ++k) d = Frag<E>::mma(__builtin_bit_cast(V, op[k]), b, d);
                if (E::CODE == SPMV_F16) {
                    const float back = ldexpf(1.0f, -e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][c][i] = fmaf(back, d[i], acc[j][c][i]);
                } else {
                    acc[j][c] = d;
                }
            }
        }
    }
    // waves add their sums one after the other, so the order is fixed
    const float f = scale ? scale[ad] : 1.0f;
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int jj = 0; jj < NJ; ++jj) {
            if (jj != j) continue;
            for (int w = 0; w < 8; ++w) {
                if (wv == w) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) sum[c][lane] = w == 0 ? acc[jj][c] : sum[c][lane] + acc[jj][c];
                }
                __syncthreads();
            }
        }
        if (wv == 0 && c0 < a.dim) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = r0 + 16 * j + 4 * q + i;
                if (row >= max_rank) break;
                float v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = row < rank ? f * sum[c][lane][i] : 0.0f;
                store_row8<F32, VEC>(a.out + ((int64_t)ad * max_rank + row) * a.dim, c0, a.dim, v);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int rank_tiles(int max_rank) { return max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : max_rank <= 64 ? 4 : 8; }

// Workgroups that share a tile's contraction: enough for 2048 workgroups in
// all, at most LR_MAX_SPLIT (the workspace's bound, which knows n_tok alone).
int max_split(int64_t n_tok) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(LR_MAX_SPLIT, 2048 / std::max<int64_t>(1, ceil_div(n_tok, LR_TILE))));
}
// ... and so that each of a workgroup's 4 waves keeps two 64-wide steps.
int split_of(int64_t n_tok, int64_t dim) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(max_split(n_tok), dim / 512));
}

size_t h_bytes(int64_t n_tok, int max_rank) {
    return ((size_t)max_split(n_tok) * (size_t)n_tok * (size_t)(16 * rank_tiles(max_rank)) * 4 + 255) & ~size_t(255);
}

spmv_status check_common(int32_t n_tok, int32_t n_in, int32_t n_out, int32_t n_adapters, int32_t max_rank,
                         int32_t dtype, const void *A, const void *B, const int32_t *order, const int32_t *offsets,
                         const int32_t *tiles, int32_t n_tiles, const void *workspace, size_t workspace_bytes) {
    if (n_tok < 0 || n_in < 1 || n_out < 1 || n_adapters < 1)
        return fail(SPMV_ERR_INVALID_VALUE, "n_tok must be >= 0, n_in, n_out and n_adapters >= 1");
    if (max_rank < 1) return fail(SPMV_ERR_INVALID_VALUE, "max_rank must be positive");
    if (max_rank > LR_MAX_RANK) return fail(SPMV_ERR_UNSUPPORTED, "ranks above %d are not supported", LR_MAX_RANK);
    if (dtype != SPMV_F16 && dtype != SPMV_BF16)
        return fail(dtype_ok(dtype) ? SPMV_ERR_UNSUPPORTED : SPMV_ERR_INVALID_VALUE, "x, A and B must be fp16 or bf16");
    int32_t want = 0;
    const spmv_status st = route_tile_count(n_tok, n_adapters, &want);
    if (st != SPMV_OK) return st;
    if (n_tiles != want)
        return fail(SPMV_ERR_INVALID_VALUE, "%d tiles, but a plan of %d tokens and %d adapters has %d", n_tiles, n_tok,
                    n_adapters, want);
    if (!A || !B || !offsets || (n_tok > 0 && (!order || !tiles))) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (!aligned16(tiles)) return fail(SPMV_ERR_UNSUPPORTED, "tiles must be 16-byte aligned");
    size_t need = 0;
    lora_workspace_size(n_tok, max_rank, &need);
    if (n_tok > 0 && !workspace) return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (lora_workspace_size gives its size)");
    if (workspace_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    return SPMV_OK;
}

bool rows16(const void *p, int64_t ld, int64_t dim, int64_t per = 8) {
    return aligned16(p) && ld % per == 0 && dim % 8 == 0;
}

template <typename F>
spmv_status by_rank(int max_rank, F f) {
    switch (rank_tiles(max_rank)) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}
template <typename F>
spmv_status by_half(int32_t dtype, F f) {
    return dtype == SPMV_F16 ? f(F16{}) : f(BF16{});
}
template <typename F>
spmv_status by_bool(bool b, F f) {
    return b ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status lora_workspace_size(int32_t n_tok, int32_t max_rank, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    if (n_tok < 0 || max_rank < 1) return fail(SPMV_ERR_INVALID_VALUE, "n_tok must be >= 0 and max_rank positive");
    if (max_rank > LR_MAX_RANK) return fail(SPMV_ERR_UNSUPPORTED, "ranks above %d are not supported", LR_MAX_RANK);
    *bytes = 2 * h_bytes(n_tok, max_rank);
    return SPMV_OK;
}

extern "C" spmv_status lora_apply(int32_t n_tok, int32_t n_in, int32_t n_out, int32_t n_adapters, int32_t max_rank,
                                  const int32_t *ranks, const float *scale, const void *A, const void *B,
                                  int32_t dtype, const int32_t *order, const int32_t *offsets, const int32_t *tiles,
                                  int32_t n_tiles, const void *x, int64_t ldx, const void *y_in, int64_t ldyin,
                                  void *y, int32_t y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    spmv_status st = check_common(n_tok, n_in, n_out, n_adapters, max_rank, dtype, A, B, order, offsets, tiles, n_tiles,
                                  workspace, workspace_bytes);
    if (st != SPMV_OK) return st;
    if (y_dtype != SPMV_F32 && y_dtype != dtype)
        return fail(dtype_ok(y_dtype) ? SPMV_ERR_UNSUPPORTED : SPMV_ERR_INVALID_VALUE, "y must be fp32 or of x's type");
    if (ldx < n_in || ldy < n_out || (y_in && ldyin < n_out))
        return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (y_in == y && y_in && ldyin != ldy) return fail(SPMV_ERR_INVALID_VALUE, "y_in is y, but their row strides differ");
    if (n_tok == 0) return SPMV_OK;
    if (!x || !y) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    hipStream_t s = as_stream(stream);
    const int split = split_of(n_tok, n_in);
    const int4 *tl = reinterpret_cast<const int4 *>(tiles);
    const ShrinkArg sa = {static_cast<const unsigned short *>(x), static_cast<const unsigned short *>(A), ldx, n_in,
                          static_cast<float *>(workspace)};
    st = by_half(dtype, [&](auto e) {
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(rows16(x, ldx, n_in) && aligned16(A), [&](auto vec) {
                k_lora_shrink<decltype(e), decltype(nj)::value, decltype(vec)::value>
                    <<<dim3(n_tiles, split, 1), 256, 0, s>>>(n_tok, n_adapters, max_rank, ranks, order, tl, sa, sa);
                SPMV_LAUNCHED("k_lora_shrink");
                return SPMV_OK;
            });
        });
    });
    if (st != SPMV_OK) return st;
    const int64_t yper = 16 / (int64_t)dtype_size(y_dtype);
    const bool vec_y = rows16(y, ldy, n_out, yper) && (!y_in || rows16(y_in, ldyin, n_out, yper)) && aligned16(B);
    const dim3 grid(n_tiles, (unsigned)ceil_div(n_out, 4 * LR_WAVE_COLS));
    return by_half(dtype, [&](auto e) {
        typedef decltype(e) E;
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(vec_y, [&](auto vec) {
                constexpr int NJ = decltype(nj)::value;
                constexpr bool VEC = decltype(vec)::value;
                auto go = [&](auto yt, auto nt) {
                    typedef decltype(yt) Y;
                    k_lora_expand<E, Y, NJ, decltype(nt)::value, VEC><<<grid, 256, 0, s>>>(
                        n_tok, n_adapters, max_rank, split, ranks, scale, order, tl, static_cast<const float *>(workspace),
                        static_cast<const unsigned short *>(B), n_out, static_cast<const typename Y::T *>(y_in), ldyin,
                        static_cast<typename Y::T *>(y), ldy);
                };
                if (y_dtype == SPMV_F32)
                    go(F32{}, std::integral_constant<int, E::CODE == SPMV_BF16 ? 3 : 2>{});
                else
                    go(E{}, std::integral_constant<int, 2>{});
                SPMV_LAUNCHED("k_lora_expand");
                return SPMV_OK;
            });
        });
    });
}

extern "C" spmv_status lora_grad(int32_t n_tok, int32_t n_in, int32_t n_out, int32_t n_adapters, int32_t max_rank,
                                 const int32_t *ranks, const float *scale, const void *A, const void *B,
                                 int32_t dtype, const int32_t *order, const int32_t *offsets, const int32_t *tiles,
                                 int32_t n_tiles, const void *x, int64_t ldx, const void *dy, int64_t lddy, float *dA,
                                 float *dB, void *workspace, size_t workspace_bytes, void *stream) {
    spmv_status st = check_common(n_tok, n_in, n_out, n_adapters, max_rank, dtype, A, B, order, offsets, tiles, n_tiles,
                                  workspace, workspace_bytes);
    if (st != SPMV_OK) return st;
    if (ldx < n_in || lddy < n_out) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (!dA || !dB || (n_tok > 0 && (!x || !dy))) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    hipStream_t s = as_stream(stream);
    const int split = split_of(n_tok, std::min(n_in, n_out));
    float *h = static_cast<float *>(workspace);
    float *g = reinterpret_cast<float *>(static_cast<char *>(workspace) + h_bytes(n_tok, max_rank));
    const auto *xs = static_cast<const unsigned short *>(x), *dys = static_cast<const unsigned short *>(dy);
    const bool vec = rows16(x, ldx, n_in) && rows16(dy, lddy, n_out) && aligned16(A) && aligned16(B) && aligned16(dA) &&
                     aligned16(dB);
    const ShrinkArg hx = {xs, static_cast<const unsigned short *>(A), ldx, n_in, h};
    const ShrinkArg gy = {dys, static_cast<const unsigned short *>(B), lddy, n_out, g};
    const OuterArg oa = {xs, ldx, n_in, (int)ceil_div(n_in, LR_WAVE_COLS), g, dA};
    const OuterArg ob = {dys, lddy, n_out, (int)ceil_div(n_out, LR_WAVE_COLS), h, dB};
    return by_half(dtype, [&](auto e) {
        typedef decltype(e) E;
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(vec, [&](auto v) {
                constexpr int NJ = decltype(nj)::value;
                constexpr bool VEC = decltype(v)::value;
                if (n_tok > 0) {
                    k_lora_shrink<E, NJ, VEC><<<dim3(n_tiles, split, 2), 256, 0, s>>>(
                        n_tok, n_adapters, max_rank, ranks, order, reinterpret_cast<const int4 *>(tiles), hx, gy);
                    SPMV_LAUNCHED("k_lora_shrink");
                }
                constexpr int JB = NJ < 4 ? NJ : 4;
                k_lora_outer<E, JB, 16 * NJ, E::CODE == SPMV_BF16 ? 3 : 2, VEC>
                    <<<dim3(oa.blocks + ob.blocks, n_adapters, NJ / JB), 512, 0, s>>>(n_tok, max_rank, split, ranks, scale, order,
                                                                             offsets, oa, ob);
                SPMV_LAUNCHED("k_lora_outer");
                return SPMV_OK;
            });
        });
    });
}
