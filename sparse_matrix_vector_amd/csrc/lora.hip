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
// h stays fp32 in memory.  As an operand it is split into a sum of 16-bit numbers.
// Three hold all 24 bits of every entry (two show where ranks cancel, bf16's 16
// bits in a rounded result too).  expand with fp16: scaled by a power of two per
// token; entries too far below the token's largest for that scale take another
// pass of the product at their own.  Otherwise, and in outer with both types:
// bf16 numbers, which need no scale.
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

// Elements c .. c + 7 of a row of n as 16 bytes.  VEC (n >= 8): one access of
// any alignment and no branch; near or past the end the row's last 8 elements,
// from n - 8 on.  Otherwise elements past the end are zero.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const unsigned short *__restrict__ row, int c, int n) {
    if (VEC) return *reinterpret_cast<const u32x4_any *>(row + min(c, n - 8));
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned int lo = row[min(c + 2 * i, n - 1)], hi = row[min(c + 2 * i + 1, n - 1)];
        r[i] = (c + 2 * i < n ? lo : 0u) | (c + 2 * i + 1 < n ? hi << 16 : 0u);
    }
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
    unsigned short *terms;         // the weight gradients' operand (below), or NULL
};

__device__ __forceinline__ int rank_of(const int *ranks, int a, int max_rank) {
    return ranks ? min(max(ranks[a], 0), max_rank) : max_rank;
}

constexpr int SHRINK_WAVES = 4;

// The token of sorted row i; whatever the plan holds, one of the batch's.
__device__ __forceinline__ int token_of(const int *__restrict__ order, int i, int n_tok) {
    return (int)min((unsigned)order[i], (unsigned)(n_tok - 1));
}

// The rows of one workgroup: a plan tile, or MT tiles of a group from every
// MT-th one on (the others of the group have nothing to do).  Workgroup `id`
// takes tile MT * (id % n) + id / n, n = tiles / MT: those with work come first
// and without gaps, or they would fall on the same compute units again and again.
struct Block {
    int group, begin, end;
};
template <int MT>
__device__ __forceinline__ Block block_of(const int4 *__restrict__ tiles, int n_tiles, int id,
                                          const int *__restrict__ offsets, int n_tok, int n_adapters) {
    if (MT > 1) {
        const int n = (n_tiles + MT - 1) / MT;
        id = MT * (id % n) + id / n;
    }
    if (id >= n_tiles) return {-1, 0, 0};
    int4 t = tiles[id];
    t.y = min(max(t.y, 0), n_tok);
    t.z = min(min(t.z, t.y + LR_TILE), n_tok);
    Block b = {(unsigned)t.x < (unsigned)n_adapters ? t.x : -1, t.y, t.z};
    if (MT > 1) {
        if ((unsigned)(t.y - t.w) % (LR_TILE * MT) != 0)
            b.end = b.begin;
        else if (t.z > t.y)
            b.end = min(min(t.y + LR_TILE * MT, n_tok), b.group >= 0 ? offsets[b.group + 1] : n_tok);
    }
    return b;
}

// v as a sum of NT numbers of type E.  bf16's first is cut off, not rounded, so that
// fp32's largest numbers stay finite (the next two still hold the 16 bits left);
// infinities and NaN are the first term alone.
template <typename E, int NT>
__device__ __forceinline__ void split_terms(float v, unsigned short (&t)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (E::CODE == SPMV_BF16 && i == 0)
            t[i] = (unsigned short)(__float_as_uint(v) >> 16);
        else
            t[i] = __builtin_bit_cast(unsigned short, (typename E::T)v);
        const float p = (float)__builtin_bit_cast(typename E::T, t[i]);
        v = i == 0 && !(fabsf(p) < INFINITY) ? 0.0f : v - p;
    }
}

// The power of two that brings max |v| = m into [2^14, 2^15), half of fp16's range
// (1 for 0, infinities and NaN), or to more than 2^-2 at least: products of fp16
// numbers are multiples of 2^-48, and the largest power leaves room to bring
// sums of the largest fp16 numbers to a smaller one's scale (2^27 columns, fp32).
__device__ __forceinline__ int scale_exponent(float m) {
    const int e = (__float_as_int(m) >> 23) & 255;
    return e == 0 || e == 255 ? 0 : min(127 + 14 - e, 46);
}
// Entries down to 2^-LR_SPREAD of the largest keep all 24 bits in three terms at that
// scale: the smallest is then 2^-1, whose last bit is fp16's, 2^-24.
constexpr int LR_SPREAD = 15;

// Operands of the weight gradients: h as three bf16 terms, 24 bits (down to bf16's
// smallest number, 2^-133) whatever its neighbours hold.  (The tokens are the
// contraction there, so a scale would have to be shared by tokens and tiles, and
// scaled fp16 terms lose what is small beside a neighbour.)  Transposed to
// [term][rank][n_tok + LR_PAD], so that 8 tokens of a rank are one load.
constexpr int LR_PAD = 8;
constexpr int LR_GRAD_TERMS = 3;
template <int R>
__device__ __forceinline__ void store_terms(unsigned short *__restrict__ terms, int n_tok, int row, int end, int rank,
                                            const float (&v)[4]) {
    unsigned short t[4][LR_GRAD_TERMS];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_terms<BF16, LR_GRAD_TERMS>(v[i], t[i]);
#pragma unroll
    for (int k = 0; k < LR_GRAD_TERMS; ++k) {
        unsigned short *p = terms + ((int64_t)k * R + rank) * (n_tok + LR_PAD) + row;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + i < end) p[i] = t[i][k];
    }
}

// The 64-wide steps lo .. hi - 1 of MT token tiles and the first N rank tiles.
// Two register sets take turns, so a step's loads are in flight over the
// previous step's products; past the end the last step is read again.
template <typename E, int N, int MT, bool VEC, int NJ>
__device__ __forceinline__ void shrink_steps(const unsigned short *const (&xr)[MT], const unsigned short *const (&wr)[NJ],
                                             int dim, int lo, int hi, int q, f32x4 (&acc)[MT][NJ]) {
    typedef typename Frag<E>::V V;
    struct Step {
        u32x4 x[MT][2], w[N][2];
    };
    auto load = [&](Step &st, int s) {
        const int k = min(s, hi - 1) * 64 + q * 16;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            st.x[m][0] = load8<VEC>(xr[m], k, dim);
            st.x[m][1] = load8<VEC>(xr[m], k + 8, dim);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            st.w[j][0] = load8<VEC>(wr[j], k, dim);
            st.w[j][1] = load8<VEC>(wr[j], k + 8, dim);
        }
    };
    auto multiply = [&](Step &st, int s) {
        if (VEC && s * 64 + 64 > dim) {
            // uniform: near the end both operands hold elements dim - 8 + e; those
            // of them that belong to an earlier piece, or that lie before this
            // one, count nothing
            const int k = s * 64 + q * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int skip = k + 8 * i - min(k + 8 * i, dim - 8);   // elements to leave out
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const unsigned int keep = (2 * d >= skip ? 0xFFFFu : 0u) | (2 * d + 1 >= skip ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int m = 0; m < MT; ++m) st.x[m][i][d] &= keep;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[m][j] = Frag<E>::mma(__builtin_bit_cast(V, st.x[m][i]), __builtin_bit_cast(V, st.w[j][i]), acc[m][j]);
    };
    if (lo >= hi) return;
    Step s0, s1;
    load(s0, lo);
    int s = lo;
    for (; s + 1 < hi; s += 2) {
        load(s1, s + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s0, s);
        load(s0, s + 2);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s1, s + 1);
    }
    if (s < hi) multiply(s0, s);
}

// h = A x (and B dy).  Bound by the reading of x once tokens abound: 8192 tokens
// of 4096 + 4096 bf16 at rank 32 30 us (134 MB, 4.4 TB/s; A and B are read again
// from L2 by every block of tokens); one token of 4096 takes 3.9 us.
// One workgroup: a block of tokens, one of `split` parts of the contraction, and
// one of `products` (the gradient needs A x and B dy).  The parts of a block are
// neighbours in the launch, so that together they read whole rows of x:
// with the blocks in front, all workgroups read the same columns of rows a
// power of two apart, which lie on few memory channels.  The waves share the range in
// runs of 64-wide steps (lane group q owns k = 16 q .. 16 q + 15 of a step, in
// x and W alike), and wave 0 adds their sums in order.
template <typename E, int NJ, int MT, bool VEC>
__global__ __launch_bounds__(64 * SHRINK_WAVES) void k_lora_shrink(int n_tok, int n_adapters, int max_rank,
                                                     const int *__restrict__ ranks,
                                                     const int *__restrict__ order, const int *__restrict__ offsets,
                                                     const int4 *__restrict__ tiles, int n_tiles, int split, int products,
                                                     ShrinkArg a0, ShrinkArg a1) {
    constexpr int WAVES = SHRINK_WAVES;
    __shared__ f32x4 part[WAVES - 1][MT][NJ][64];
    const int id = blockIdx.x / split, spl = blockIdx.x - id * split;
    const int tile = products > 1 ? id >> 1 : id;
    const ShrinkArg &a = products > 1 && (id & 1) ? a1 : a0;
    const Block blk = block_of<MT>(tiles, n_tiles, tile, offsets, n_tok, n_adapters);
    if (blk.group < 0 || blk.begin >= blk.end) return;
    const int rank = rank_of(ranks, blk.group, max_rank);
    const int nj = (rank + 15) / 16;
    if (nj == 0) return;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const unsigned short *xr[MT], *wr[NJ];
#pragma unroll
    for (int m = 0; m < MT; ++m) xr[m] = a.x + (int64_t)token_of(order, min(blk.begin + 16 * m + n, blk.end - 1), n_tok) * a.ldx;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        wr[j] = a.W + ((int64_t)blk.group * max_rank + min(16 * j + n, max_rank - 1)) * a.dim;
    // steps of this wave: waves of all splits take contiguous runs of 64-wide steps
    const int steps = (a.dim + 63) / 64, parts = split * WAVES, mine = spl * WAVES + wv;
    const int lo = (int)((int64_t)steps * mine / parts), hi = (int)((int64_t)steps * (mine + 1) / parts);
    f32x4 acc[MT][NJ];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[m][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the rank tiles in use decide the loop, so that no load is conditional
    if (NJ <= 4 || nj <= NJ / 2) {
        if (NJ >= 4 && nj > 3)
            shrink_steps<E, NJ < 4 ? NJ : 4, MT, VEC>(xr, wr, a.dim, lo, hi, q, acc);
        else if (NJ >= 4 && nj > 2)
            shrink_steps<E, NJ < 3 ? NJ : 3, MT, VEC>(xr, wr, a.dim, lo, hi, q, acc);
        else if (NJ >= 2 && nj > 1)
            shrink_steps<E, NJ < 2 ? NJ : 2, MT, VEC>(xr, wr, a.dim, lo, hi, q, acc);
        else
            shrink_steps<E, 1, MT, VEC>(xr, wr, a.dim, lo, hi, q, acc);
    } else {
        shrink_steps<E, NJ, MT, VEC>(xr, wr, a.dim, lo, hi, q, acc);
    }
    if (wv > 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NJ; ++j) part[wv - 1][m][j][lane] = acc[m][j];
    }
    __syncthreads();
    if (wv > 0) return;
    float *h = a.h + (int64_t)spl * n_tok * (16 * NJ);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row0 = blk.begin + 16 * m + 4 * q;    // D: row 4 q + i, column n
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
            for (int w = 0; w < WAVES - 1; ++w) acc[m][j] += part[w][m][j][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * j + n >= rank || row0 + i >= blk.end) acc[m][j][i] = 0.0f;
        }
        if (!a.terms) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row0 + i < blk.end) h[(int64_t)(row0 + i) * (16 * NJ) + 16 * j + n] = acc[m][j][i];
            continue;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float v[4] = {acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]};
            store_terms<16 * NJ>(a.terms, n_tok, row0, blk.end, 16 * j + n, v);
        }
    }
}

// Adds a split shrink's parts in order and writes the gradients' operands:
// one wave per tile and product.
template <int NJ>
__global__ __launch_bounds__(64) void k_lora_terms(int n_tok, int n_adapters, int max_rank, int split,
                                                   const int *__restrict__ ranks,
                                                   const int4 *__restrict__ tiles, ShrinkArg a0, ShrinkArg a1) {
    constexpr int R = 16 * NJ;
    const ShrinkArg &a = blockIdx.y ? a1 : a0;
    int4 tile = tiles[blockIdx.x];
    tile.y = min(max(tile.y, 0), n_tok);
    tile.z = min(min(tile.z, tile.y + LR_TILE), n_tok);
    if ((unsigned)tile.x >= (unsigned)n_adapters || tile.y >= tile.z) return;
    if (rank_of(ranks, tile.x, max_rank) == 0) return;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int row0 = tile.y + 4 * q;
    float v[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = min(row0 + i, tile.z - 1);
            float t = 0.0f;
            for (int s = 0; s < split; ++s) t += a.h[((int64_t)s * n_tok + row) * R + 16 * j + n];
            v[j][i] = row0 + i < tile.z ? t : 0.0f;
        }
#pragma unroll
    for (int j = 0; j < NJ; ++j) store_terms<R>(a.terms, n_tok, row0, tile.z, 16 * j + n, v[j]);
}

// Eight neighbouring results of one token, read and written once (non-temporal:
// 4093 tokens of 12288 bf16 results, inputs from HBM, 75.6 against 81.8 us).
// VEC (n >= 8): near the end the row's last 8; a lane whose columns overlap its
// neighbour's stores its own only.
template <typename Y>
struct RowPiece {
    typename Y::T v[8];
};
template <typename Y, bool VEC>
__device__ __forceinline__ void load_piece(RowPiece<Y> &r, const typename Y::T *p, int c, int n) {
    if (VEC) {
        constexpr int PER = 16 / (int)sizeof(typename Y::T);
#pragma unroll
        for (int i = 0; i < 8; i += PER) {
            const Vec<Y, PER> t = load_once<Y, PER>(p + min(c, n - 8) + i);
#pragma unroll
            for (int k = 0; k < PER; ++k) r.v[i + k] = t.v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = p[min(c + i, n - 1)];
    }
}
template <typename Y, bool VEC>
__device__ __forceinline__ void store_row8(typename Y::T *p, int c, int n, const float (&v)[8]) {
    if (VEC && c + 8 <= n) {
        constexpr int PER = 16 / (int)sizeof(typename Y::T);
#pragma unroll
        for (int i = 0; i < 8; i += PER) {
            Vec<Y, PER> r;
#pragma unroll
            for (int k = 0; k < PER; ++k) r.v[k] = (typename Y::T)v[i + k];
            store_once<Y, PER>(p + c + i, r);
        }
    } else {
        const int at = VEC ? n - 8 : c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i >= c && at + i < n) p[at + i] = (typename Y::T)v[i];
    }
}

// Bound by the traffic of y and B: 4093 tokens of 12288 bf16 results at rank 64, read
// and written, 201 MB in 51 us (3.9 TB/s), and 412 MB of B from L2, which every tile
// of tokens reads for itself.
// One workgroup: a tile of tokens and 512 columns, 128 per wave; the columns
// of a tile are neighbours in the launch and together move whole rows of y.
// Two or four tiles per workgroup, sharing B, were slower (79 and 114 us against
// 67 then): fewer rows in flight.
// fp16's third term and its passes by size (normal entries: a second one in 6e-5 of
// them, so 1 tile in 8 at rank 128) cost 4 to 5 %, 12 at rank 128 (3000 tokens of
// 2048 columns, 8192 fp16 results: 66.5 us; 59.4 with small entries lost).  Such
// tiles in fp32 on the vector unit instead: 91.6.  Two passes in every tile (rows
// of A 8 times apart; 4093 tokens, rank 64, 12288 fp16 results): 125 us, 104 with one.
template <typename E, typename Y, int NJ, bool VEC>
__global__ __launch_bounds__(256, VEC ? 3 : 1) void k_lora_expand(int n_tok, int n_adapters, int max_rank, int split,
                                                     const int *__restrict__ ranks,
                                                     const float *__restrict__ scale,
                                                     const int *__restrict__ order, const int *__restrict__ offsets,
                                                     const int4 *__restrict__ tiles, int n_tiles, const float *__restrict__ h,
                                                     const unsigned short *__restrict__ B, int dim, int pieces,
                                                     const typename Y::T *y_in, int64_t ldyin,
                                                     typename Y::T *y, int64_t ldy) {
    typedef typename Frag<E>::V V;
    constexpr int R = 16 * NJ, LD = R + 8;
    constexpr bool F = E::CODE == SPMV_F16;
    constexpr int NT = 3;
    __shared__ __attribute__((aligned(16))) unsigned short hs[NT][LR_TILE][LD];
    __shared__ int exps[LR_TILE], again[4];
    const int id = blockIdx.x / pieces, piece = blockIdx.x - id * pieces;
    const Block blk = block_of<1>(tiles, n_tiles, id, offsets, n_tok, n_adapters);
    if (blk.begin >= blk.end) return;
    const int rank = blk.group >= 0 ? rank_of(ranks, blk.group, max_rank) : 0;
    if (rank == 0 && y_in == y) return;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int c0 = piece * (4 * LR_WAVE_COLS) + wv * LR_WAVE_COLS + 8 * n;

    // y_in of the lane's rows is in flight over everything else
    int64_t tok[4];
    RowPiece<Y> base[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) tok[i] = token_of(order, min(blk.begin + 4 * q + i, blk.end - 1), n_tok);
    if (y_in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) load_piece<Y, VEC>(base[i], y_in + tok[i] * ldyin, c0, dim);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 8; ++c) base[i].v[c] = (typename Y::T)0.0f;
    }
    f32x4 acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int e[4] = {0, 0, 0, 0};
    if (rank > 0) {
        const unsigned short *Br = B + (int64_t)blk.group * max_rank * dim;
        u32x4 r[8];
        auto load_b = [&](int jb) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = load8<VEC>(Br + (int64_t)min(jb + i, max_rank - 1) * dim, c0, dim);
        };
        load_b(NJ == 1 ? 8 * (q & 1) : 8 * q);
        // 16 lanes per token: the partial sums of h in order
        const int t = (threadIdx.x >> 4), l = threadIdx.x & 15;
        const int64_t row = min(blk.begin + t, blk.end - 1);
        float v[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) v[j] = 0.0f;
        const float *hr = h + row * R + l;
#pragma unroll 4
        for (int s = 0; s < split; ++s)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (16 * j < rank) v[j] += hr[(int64_t)s * n_tok * R + 16 * j];
        // The terms of v.  fp16: of the entries that are not far below the token's
        // largest, at the scale of that; the others stay in v for another pass.
        auto next_terms = [&]() {
            int e = 0;
            float least = 0.0f;
            if (F) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) top = fmaxf(top, fabsf(v[j]));
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
                e = scale_exponent(top);
                least = ldexpf(top, -LR_SPREAD);
            }
            bool left = false;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float now = v[j];
                if (F) {
                    const bool later = fabsf(now) < least;
                    left |= later && now != 0.0f;
                    v[j] = later ? now : 0.0f;
                    now = later ? 0.0f : ldexpf(now, e);
                }
                unsigned short terms[NT];
                split_terms<E, NT>(now, terms);
#pragma unroll
                for (int i = 0; i < NT; ++i) hs[i][t][16 * j + l] = terms[i];
            }
            if (F) {
                if (l == 0) exps[t] = e;
                const int any = __any(left);
                if (lane == 0) again[wv] = any;
            }
            __syncthreads();
        };
        // acc += the terms times B; loaded: r holds B's first rows
        auto multiply = [&](bool loaded) {
            if constexpr (NJ == 1) {
                // up to 16 ranks: the terms share the contraction, eight ranks
                // of one term per lane group and step
                constexpr int STEPS = (2 * NT + 3) / 4;
                const int live = rank - 8 * (q & 1);
                if (!loaded) load_b(8 * (q & 1));
                if (rank < 16) {                            // rows past the rank may hold anything
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int w = 0; w < 4; ++w) r[i][w] = i < live ? r[i][w] : 0u;
                }
                V a[STEPS];
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int term = 2 * s + (q >> 1);
                    u32x4 w = {0u, 0u, 0u, 0u};
                    if (term < NT)
                        w = *reinterpret_cast<const u32x4 *>(&hs[term < NT ? term : 0][n][8 * (q & 1)]);
                    a[s] = __builtin_bit_cast(V, w);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const V b = __builtin_bit_cast(V, column_of(r, c));
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) acc[c] = Frag<E>::mma(a[s], b, acc[c]);
                }
            } else {
                for (int j0 = 0; j0 < rank; j0 += 32) {
                    const int jb = j0 + 8 * q;
                    if (j0 > 0 || !loaded) load_b(jb);
                    if (j0 + 32 > rank) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int w = 0; w < 4; ++w) r[i][w] = jb + i < rank ? r[i][w] : 0u;
                    }
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
        };
        for (bool first = true;; first = false) {
            next_terms();
            if (F) {
                // the sums so far to this pass's scale
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int to = exps[4 * q + i];
                    if (!first) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) acc[c][i] = ldexpf(acc[c][i], to - e[i]);
                    }
                    e[i] = to;
                }
            }
            multiply(first);
            // uniform; rare for entries of ordinary spread, and 8 passes at most for sums
            // of fp16 products, as each takes every token's entries of 15 powers of two
            if (!F || !(again[0] | again[1] | again[2] | again[3])) break;
            __syncthreads();
        }
    }
    if (c0 >= dim) return;
    const float f = rank > 0 && scale ? scale[blk.group] : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * q + i;
        if (blk.begin + t >= blk.end) break;
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = (float)base[i].v[c];
        if (rank > 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = fmaf(f, F ? ldexpf(acc[c][i], -e[i]) : acc[c][i], v[c]);
        }
        store_row8<Y, VEC>(y + tok[i] * ldy, c0, dim, v);
    }
}

// Eight elements as an exact sum of N operands in bf16: fp16's 11 bits are one
// number of 8 and one of 3, and bf16 holds all of its exponents.  For fp16 this
// conversion, on the vector unit and once per reading of x, costs 2 to 10 us: 8192
// tokens, 4096 + 4096 columns, rank 32, 4 adapters 69 us a gradient against 62 with
// h as scaled fp16 numbers, which dropped entries 2^25 below their neighbours;
// 2048 + 2048 columns, 1 adapter, 85 against 60.  Without the smallest of the six
// products 2 % less.
template <typename E>
struct Exact;
template <>
struct Exact<BF16> {
    static constexpr int N = 1;
    b8 v[N];
    __device__ __forceinline__ explicit Exact(u32x4 r) { v[0] = __builtin_bit_cast(b8, r); }
};
template <>
struct Exact<F16> {
    static constexpr int N = 2;
    b8 v[N];
    __device__ __forceinline__ explicit Exact(u32x4 r) {
        const h8 h = __builtin_bit_cast(h8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (float)h[i];
            v[0][i] = (__bf16)f;
            v[1][i] = (__bf16)(f - (float)v[0][i]);
        }
    }
};

struct OuterArg {
    const unsigned short *x;   // x or dy
    int64_t ldx;
    int dim, blocks;           // columns, and their 128-column blocks
    const unsigned short *terms;
    float *out;                // [n_adapters, max_rank, dim]
};

// Bound by the latency of the rows of x and dy, which few waves walk (a
// workgroup has one adapter's 128 columns): 8192 tokens of 4096 + 4096 bf16,
// rank 32, 4 adapters 38 us (134 MB, 3.5 TB/s); 300 fp16 tokens at rank 8 6.2 us.
// More workgroups would have to add partial gradients; the terms loaded a step
// ahead as well was 3 to 8 % slower (registers).
// One workgroup: 128 columns of adapter blockIdx.y's gradient; blockIdx.x
// counts the column blocks of the first product, then of the second, and
// blockIdx.z blocks of NJ rank tiles out of the R / 16 of h.  The waves take
// turns over 32-token steps (two plan tiles), the next step's rows loading
// over the current one's products, and their sums are added in order, each wave
// those of its own columns.
template <typename E, int NJ, int R, int WAVES, bool VEC>
__global__ __launch_bounds__(64 * WAVES) void k_lora_outer(int n_tok, int max_rank,
                                                    const int *__restrict__ ranks,
                                                    const float *__restrict__ scale,
                                                    const int *__restrict__ order,
                                                    const int *__restrict__ offsets, OuterArg a0, OuterArg a1) {
    constexpr int NT = LR_GRAD_TERMS;
    __shared__ f32x4 sum[WAVES][8][64];
    const int r0 = blockIdx.z * 16 * NJ;   // first rank of this workgroup
    const bool second = (int)blockIdx.x >= a0.blocks;
    const OuterArg &a = second ? a1 : a0;
    const int ad = blockIdx.y;
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int c0 = (blockIdx.x - (second ? a0.blocks : 0)) * LR_WAVE_COLS + 8 * n;
    const int rank = rank_of(ranks, ad, max_rank);
    const int t0 = min(max(offsets[ad], 0), n_tok), t1 = rank > r0 ? min(max(offsets[ad + 1], t0), n_tok) : t0;
    f32x4 acc[NJ][8];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int tok[8];
    auto load_tok = [&](int t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) tok[i] = token_of(order, min(t + 8 * q + i, t1 - 1), n_tok);
    };
    auto load_rows = [&](u32x4(&r)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = load8<VEC>(a.x + (int64_t)tok[i] * a.ldx, c0, a.dim);
    };
    auto step = [&](int t, u32x4(&r)[8], u32x4(&next)[8]) {
        // the next step's rows, and the tokens of the one after (past the end
        // the last ones again)
        load_rows(next);
        load_tok(t + 64 * WAVES);
        __builtin_amdgcn_sched_barrier(0);
        const int at = min(t + 8 * q, t1 - 1), valid = t1 - (t + 8 * q);   // tokens of this lane
        u32x4 op[NJ][NT];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int k = 0; k < NT; ++k)
                __builtin_memcpy(&op[j][k], a.terms + ((int64_t)k * R + r0 + 16 * j + n) * (n_tok + LR_PAD) + at, 16);
        if (t + 32 > t1) {                 // uniform: tokens past the end count nothing
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        op[j][k][d] = valid > 2 * d + 1 ? op[j][k][d] : valid > 2 * d ? op[j][k][d] & 0xFFFFu : 0u;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const Exact<E> b(column_of(r, c));
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    const b8 g = __builtin_bit_cast(b8, op[j][k]);
#pragma unroll
                    for (int i = 0; i < Exact<E>::N; ++i) acc[j][c] = Frag<BF16>::mma(g, b.v[i], acc[j][c]);
                }
        }
    };
    int t = t0 + 32 * wv;
    if (t < t1) {
        u32x4 ra[8], rb[8];
        load_tok(t);
        load_rows(ra);
        load_tok(t + 32 * WAVES);
        for (; t < t1; t += 64 * WAVES) {
            step(t, ra, rb);
            if (t + 32 * WAVES < t1) step(t + 32 * WAVES, rb, ra);
        }
    }
    // the waves' sums, in wave order, shared out over the waves by product
    const float f = scale ? scale[ad] : 1.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[wv][c][lane] = acc[j][c];
        __syncthreads();
#pragma unroll
        for (int c = wv; c < 8; c += WAVES) {
            f32x4 all = sum[0][c][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) all += sum[w][c][lane];
            sum[0][c][lane] = all;
        }
        __syncthreads();
        // wave w writes the rows 4 q + (w & 3), of 8 waves those of half the lanes' groups
        const int i = wv & 3;
        const int row = r0 + 16 * j + 4 * q + i;
        if ((WAVES == 4 || (q & 1) == (wv >> 2)) && row < max_rank && c0 < a.dim) {
            float v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const f32x4 s4 = sum[0][c][lane];
                const float s1 = i == 0 ? s4[0] : i == 1 ? s4[1] : i == 2 ? s4[2] : s4[3];
                v[c] = row < rank ? f * s1 : 0.0f;
            }
            store_row8<F32, VEC>(a.out + ((int64_t)ad * max_rank + row) * a.dim, c0, a.dim, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int rank_tiles(int max_rank) { return max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : max_rank <= 64 ? 4 : 8; }

constexpr int LR_WIDE = 4;

// lora_grad's products take blocks of LR_WIDE tiles, an operand of A or B serving
// all of them, where that still fills the card and adapters have 64 tokens or
// more on average.  Gradient in us with (and without), bf16; fp16 the same way:
//   tokens                          4096         6000         8192        16384
//   4 adapters, 4096^2, rank 32  46.2 (44.7)  79.1 (63.3)  60.8 (81.1)  116 (154)
//   1 adapter,  2048^2, rank 32  43.1 (41.3)  53.8 (57.6)  63.9 (73.3)  131 (152)
//   4 adapters, 4096^2, rank 16  40.2 (35.5)  66.9 (49.7)  56.0 (65.1)  106 (123)
//   8 adapters, 4096^2, rank 16                            90   (70)    121 (126)
// Up to rank 16 and below 16384 tokens it depends on the number of adapters.
// At rank 64 the registers do not allow it.  lora_apply is better off with single
// tiles (8192 tokens 69 us, 82 in blocks).
bool wide_blocks(int64_t n_tok, int64_t n_adapters, int max_rank) {
    return max_rank <= 32 && n_tok >= 64 * n_adapters && n_tok >= (max_rank <= 16 ? 16384 : 8192);
}

// Workgroups that share a block's contraction.  Whoever reads h adds the parts,
// once per 512 columns of the result, so there are only as many as it takes to
// have LR_FILL workgroups, each wave with at least two 64-wide steps.  The
// workspace holds the most that n_tok alone allows.
constexpr int LR_FILL = 256;
int max_split(int64_t n_tok) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(LR_MAX_SPLIT, LR_FILL / std::max<int64_t>(1, ceil_div(n_tok, LR_TILE))));
}
int split_of(int64_t n_tok, int64_t blocks, int64_t dim) {
    const int64_t fill = std::min<int64_t>(max_split(n_tok), ceil_div(LR_FILL, std::max<int64_t>(1, blocks)));
    return (int)std::max<int64_t>(1, std::min<int64_t>(fill, dim / (128 * SHRINK_WAVES)));
}

size_t h_bytes(int64_t n_tok, int max_rank) {
    return ((size_t)max_split(n_tok) * (size_t)n_tok * (size_t)(16 * rank_tiles(max_rank)) * 4 + 255) & ~size_t(255);
}
// terms of one product
size_t terms_bytes(int64_t n_tok, int max_rank) {
    return ((size_t)LR_GRAD_TERMS * (size_t)(16 * rank_tiles(max_rank)) * (size_t)(n_tok + LR_PAD) * 2 + 255) & ~size_t(255);
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
    if (n_tok > 0) lora_workspace_size(n_tok, max_rank, &need);
    if (n_tok > 0 && !workspace) return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (lora_workspace_size gives its size)");
    if (workspace_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    return SPMV_OK;
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
    *bytes = 2 * (h_bytes(n_tok, max_rank) + terms_bytes(n_tok, max_rank));
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
    const int64_t pieces = ceil_div(n_out, 4 * LR_WAVE_COLS);
    st = check_grid(n_tiles * pieces);
    if (st != SPMV_OK) return st;
    const int grid = (int)(n_tiles * pieces);
    hipStream_t s = as_stream(stream);
    const int split = split_of(n_tok, n_tiles, n_in);
    const int4 *tl = reinterpret_cast<const int4 *>(tiles);
    const ShrinkArg sa = {static_cast<const unsigned short *>(x), static_cast<const unsigned short *>(A), ldx, n_in,
                          static_cast<float *>(workspace), nullptr};
    st = by_half(dtype, [&](auto e) {
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(n_in >= 8, [&](auto vec) {
                constexpr int NJ = decltype(nj)::value;
                constexpr bool VEC = decltype(vec)::value;
                k_lora_shrink<decltype(e), NJ, 1, VEC><<<n_tiles * split, 64 * SHRINK_WAVES, 0, s>>>(
                    n_tok, n_adapters, max_rank, ranks, order, offsets, tl, n_tiles, split, 1, sa, sa);
                SPMV_LAUNCHED("k_lora_shrink");
                return SPMV_OK;
            });
        });
    });
    if (st != SPMV_OK) return st;
    return by_half(dtype, [&](auto e) {
        typedef decltype(e) E;
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(n_out >= 8, [&](auto vec) {
                constexpr int NJ = decltype(nj)::value;
                constexpr bool VEC = decltype(vec)::value;
                auto go = [&](auto yt) {
                    typedef decltype(yt) Y;
                    k_lora_expand<E, Y, NJ, VEC><<<grid, 256, 0, s>>>(
                        n_tok, n_adapters, max_rank, split, ranks, scale, order, offsets, tl, n_tiles,
                        static_cast<const float *>(workspace), static_cast<const unsigned short *>(B), n_out,
                        (int)pieces,
                        static_cast<const typename Y::T *>(y_in), ldyin, static_cast<typename Y::T *>(y), ldy);
                };
                if (y_dtype == SPMV_F32)
                    go(F32{});
                else
                    go(E{});
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
    const bool wide = wide_blocks(n_tok, n_adapters, max_rank);
    const int split = split_of(n_tok, 2 * n_tiles, std::min(n_in, n_out));   // 1 in wide blocks: n_tok alone sees to it
    const size_t hb = h_bytes(n_tok, max_rank), tb = terms_bytes(n_tok, max_rank);
    char *w = static_cast<char *>(workspace);
    const auto *xs = static_cast<const unsigned short *>(x), *dys = static_cast<const unsigned short *>(dy);
    const bool vec = n_in >= 8 && n_out >= 8;
    const int4 *tl = reinterpret_cast<const int4 *>(tiles);
    unsigned short *terms[2];
    for (int i = 0; i < 2; ++i) terms[i] = reinterpret_cast<unsigned short *>(w + 2 * hb + i * tb);
    ShrinkArg hx = {xs, static_cast<const unsigned short *>(A), ldx, n_in, reinterpret_cast<float *>(w), terms[0]};
    ShrinkArg gy = {dys, static_cast<const unsigned short *>(B), lddy, n_out, reinterpret_cast<float *>(w + hb), terms[1]};
    const OuterArg oa = {xs, ldx, n_in, (int)ceil_div(n_in, LR_WAVE_COLS), terms[1], dA};
    const OuterArg ob = {dys, lddy, n_out, (int)ceil_div(n_out, LR_WAVE_COLS), terms[0], dB};
    return by_half(dtype, [&](auto e) {
        typedef decltype(e) E;
        return by_rank(max_rank, [&](auto nj) {
            return by_bool(vec, [&](auto v) {
                constexpr int NJ = decltype(nj)::value;
                constexpr bool VEC = decltype(v)::value;
                if (n_tok > 0) {
                    ShrinkArg s0 = hx, s1 = gy;
                    if (split > 1) s0.terms = s1.terms = nullptr;
                    if (NJ <= 2 && wide) {
                        constexpr int MT = NJ <= 2 ? LR_WIDE : 1;
                        k_lora_shrink<E, NJ, MT, VEC><<<(n_tiles + MT - 1) / MT * MT * split * 2, 64 * SHRINK_WAVES, 0, s>>>(
                            n_tok, n_adapters, max_rank, ranks, order, offsets, tl, n_tiles, split, 2, s0, s1);
                    } else {
                        k_lora_shrink<E, NJ, 1, VEC><<<n_tiles * split * 2, 64 * SHRINK_WAVES, 0, s>>>(
                            n_tok, n_adapters, max_rank, ranks, order, offsets, tl, n_tiles, split, 2, s0, s1);
                    }
                    SPMV_LAUNCHED("k_lora_shrink");
                    if (split > 1) {
                        k_lora_terms<NJ><<<dim3(n_tiles, 2), 64, 0, s>>>(n_tok, n_adapters, max_rank, split, ranks, tl, hx,
                                                                           gy);
                        SPMV_LAUNCHED("k_lora_terms");
                    }
                }
                // With few column blocks, 8 waves and one rank tile per workgroup fill
                // the card better; with more, 4 waves, so that two workgroups share a
                // CU, and two rank tiles that share a reading of x.  Gradient in us with 8
                // waves and one rank tile (with 4 and, above rank 16, two), bf16; fp16 alike:
                //   blocks     32          64          128         192         256
                //   rank 16 65.6 (81.4) 19.8 (20.5) 23.0 (24.5) 27.8 (27.6) 34.0 (35.9)
                //   rank 32 64.1 (88.5) 23.1 (26.6) 28.4 (31.4) 42.1 (40.0) 53.9 (44.5)
                //   rank 64 91.4 (115)  29.4 (32.8) 46.4 (41.2) 66.2 (59.6) 92.8 (68.7)
                // (32 blocks: 8192 tokens, otherwise 4096).  Above rank 32 the two meet
                // nearer 100 blocks.
                constexpr int JB = NJ < 2 ? NJ : 2;
                const int64_t blocks = (int64_t)(oa.blocks + ob.blocks) * n_adapters;
                if (blocks < 192)
                    k_lora_outer<E, 1, 16 * NJ, 8, VEC><<<dim3(oa.blocks + ob.blocks, n_adapters, NJ), 64 * 8, 0, s>>>(
                        n_tok, max_rank, ranks, scale, order, offsets, oa, ob);
                else
                    k_lora_outer<E, JB, 16 * NJ, 4, VEC><<<dim3(oa.blocks + ob.blocks, n_adapters, NJ / JB), 64 * 4, 0, s>>>(
                        n_tok, max_rank, ranks, scale, order, offsets, oa, ob);
                SPMV_LAUNCHED("k_lora_outer");
                return SPMV_OK;
            });
        });
    });
}
