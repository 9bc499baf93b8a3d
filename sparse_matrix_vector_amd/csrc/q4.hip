// Products with 4-bit weights on gfx950: y[t, :] = alpha * W x[t, :] + beta * y[t, :].
//
// The codes go from memory straight to the registers that decode them, and the
// matrix cores serve one token as well as 16: the product of a fragment costs the
// same, and decoding is what the vector unit does.  Up to 4 tokens (k_q4_few) the
// waves of a workgroup split the columns of 16 rows and the bound is HBM; up to 64 of
// smaller weights (k_q4_mid) they also bring x themselves; more (k_q4_tile) share
// tiles of x through LDS.
//
// Measured, a pass among others, with what the bytes take at the rate of a large copy
// (5.2 TB/s) or the products at the rate of a large fp16 product (1.15 PFLOP/s): 12288 x
// 12288, one token 14.9 us (15.0; reads alone reach 7.1 TB/s here), 48 tokens 35 to 37
// (16), 513 tokens 185 to 190 (135); 5003 x 4100 in groups of 32 with zero points, 7
// tokens 7.8 (2.4); 2048 x 2048, one token 6.8, of which the GPU has 3.5.  A kernel trace
// has the kernels longer: k_q4_mid 8.4 to 8.8 for the 7 tokens, k_q4_tile 204 to 207 for
// the 513.
#include "q4.hpp"

#include <algorithm>

namespace spmv {
namespace {

constexpr int QF_UNROLL = 2;         // blocks of a wave's turn
constexpr int QF_AHEAD = 1;          // turns whose codes are on their way
constexpr int QF_WAVES = 8;
constexpr int QF_TOKENS = 4;
// Bytes of x at most, so that a CU has two workgroups.  With 128 KB (f16, groups of 128)
// 3 tokens of 4096 x 12288 take 8.4 us against 10.4 by tiles, but 4 tokens of 12288 x
// 12288 25.4 against 19.4.
constexpr int QF_LDS = 65536;

template <class E>
__device__ __forceinline__ void q4_store(void *y, bool f32, int64_t at, float v, float beta) {
    if (f32) {
        float *p = static_cast<float *>(y) + at;
        *p = beta != 0.0f ? fmaf(beta, *p, v) : v;
    } else {
        typename E::T *p = static_cast<typename E::T *>(y) + at;
        *p = (typename E::T)(beta != 0.0f ? fmaf(beta, (float)*p, v) : v);
    }
}

// Up to TP tokens: a workgroup owns 16 rows and keeps x whole in LDS (padded with
// zeros to whole blocks); its waves take QF_UNROLL blocks in turn, whose codes are
// loaded QF_AHEAD turns before they are used.  12288 x 12288, one token: 77.9 MB in 14
// us, 5.4 TB/s, bound by HBM (24 us with x from memory in every wave); three turns
// ahead took as long as one.
template <class E, bool ZP, int G, int TP>
__global__ __launch_bounds__(64 * QF_WAVES) void k_q4_few(int n_rows, int n_cols, int n_blk,
                                                              const char *__restrict__ tiles, int n_tok, float alpha,
                                                              const typename E::T *__restrict__ x, int64_t ldx,
                                                              float beta, void *__restrict__ y, bool f32, int64_t ldy) {
    constexpr int U = QF_UNROLL, A = QF_AHEAD, GB = Q4_BLOCK / G, PG = G / 32;
    extern __shared__ __attribute__((aligned(16))) u32x4 lds[];       // x [n_tok][ld], then the waves' sums
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int quarter = lane / 16;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int ld = n_blk * 16 + 1;                  // 16-byte pieces of a token: the odd one spreads tokens over the banks
    const Q4Rows<ZP, G> row(tiles, blockIdx.x, n_blk);
    Q4Piece<E, ZP, G> w[A + 1][U];
    const int step = waves * U;
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
        for (int u = 0; u < U; ++u) w[a][u].load(row, min(wv * U + a * step + u, n_blk - 1));
    for (int i = threadIdx.x; i < n_tok * n_blk * 16; i += blockDim.x) {
        const int t = TP == 1 ? 0 : i / (n_blk * 16), p = i - t * n_blk * 16;
        lds[t * ld + p] = q4_token_piece(x + t * ldx, (int64_t)p * 8, n_cols);
    }
    __syncthreads();
    // tokens past the end take the last one's row: their sums are not stored
    const u32x4 *xr = lds + (TP == 1 ? 0 : min(lane & 15, n_tok - 1) * ld) + quarter;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = wv * U; b0 < n_blk; b0 += (A + 1) * step) {
#pragma unroll
        for (int a = 0; a <= A; ++a) {
            const int b = b0 + a * step;
#pragma unroll
            for (int u = 0; u < U; ++u) w[(a + A) % (A + 1)][u].load(row, min(b + A * step + u, n_blk - 1));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (b + u >= n_blk) break;
#pragma unroll
                for (int g = 0; g < GB; ++g) {
                    const typename Q4Op<E>::Zero nz = Q4Op<E>::zero(w[a][u].zero(g));
                    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int m = g * PG; m < (g + 1) * PG; ++m)
                        sum = Q4Op<E>::mfma(xr[(b + u) * 16 + 4 * m], Q4Op<E>::decode(w[a][u].c[m], nz), sum);
                    const float s = w[a][u].scale(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, sum[i], acc[i]);
                }
            }
        }
    }
    __syncthreads();
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);
    part[wv * 64 + lane] = acc;
    __syncthreads();
    const float *sums = reinterpret_cast<const float *>(lds);
    for (int o = threadIdx.x; o < 16 * n_tok; o += blockDim.x) {
        const int r = o % 16, t = o / 16, at = ((t / 4) * 16 + r) * 4 + t % 4;
        float v = 0.0f;
        for (int k = 0; k < waves; ++k) v += sums[k * 256 + at];
        if (row0 + r < n_rows) q4_store<E>(y, f32, t * ldy + row0 + r, Q4Op<E>::UNIT * (alpha * v), beta);
    }
}

// Up to 64 tokens of smaller weights: as above, for 16 TT tokens, but a wave brings x
// block by block into LDS of its own (16-byte pieces exchanged within a row by the
// token's number, so that 16 tokens' pieces lie in different banks): no waiting for
// other waves before the sums at the end.  Bound by the latency of a chain of 4 or 5
// loads, since a wave has one block ahead, where there are few blocks (5003 x 4100, 7
// tokens: 13 MB in 7.8 us), by x from L2, once for every 16 rows, where there are many
// (4096 x 4096, 48 tokens: 101 MB of x and 9 of weights in 9.8 us).
template <class E, bool ZP, int G, int TT>
__global__ __launch_bounds__(64 * QF_WAVES) void k_q4_mid(int n_rows, int n_cols, int n_blk,
                                                          const char *__restrict__ tiles, int n_tok, float alpha,
                                                          const typename E::T *__restrict__ x, int64_t ldx, float beta,
                                                          void *__restrict__ y, bool f32, int64_t ldy) {
    constexpr int PG = G / 32, TN = 16 * TT;
    extern __shared__ __attribute__((aligned(16))) u32x4 lds[];       // [waves][TN][16], then the waves' sums
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int quarter = lane / 16;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const Q4Rows<ZP, G> row(tiles, blockIdx.x, n_blk);
    u32x4 *mine = lds + wv * TN * 16;
    const int piece = lane % 16;
    const typename E::T *xr[4 * TT];                 // tokens past the end take the last one's row
#pragma unroll
    for (int q = 0; q < 4 * TT; ++q) xr[q] = x + (int64_t)min(4 * q + quarter, n_tok - 1) * ldx;
    auto load_x = [&](int b, u32x4 (&v)[4 * TT]) {
#pragma unroll
        for (int q = 0; q < 4 * TT; ++q) v[q] = q4_token_ahead(xr[q], b * Q4_BLOCK + piece * 8, n_cols);
    };
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Q4Piece<E, ZP, G> w[2];
    u32x4 v[4 * TT];
    load_x(min(wv, n_blk - 1), v);
    w[0].load(row, min(wv, n_blk - 1));
    for (int bb = wv; bb < n_blk; bb += 2 * waves) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int b = bb + a * waves;
            if (b >= n_blk) break;
            if (b == n_cols / Q4_BLOCK) {
#pragma unroll
                for (int q = 0; q < 4 * TT; ++q) v[q] = q4_token_placed(v[q], b * Q4_BLOCK + piece * 8, n_cols);
            }
            wave_lds_order();                        // after the reads of the block before
#pragma unroll
            for (int q = 0; q < 4 * TT; ++q) {
                const int t = 4 * q + quarter;
                mine[t * 16 + (piece ^ (t & 15))] = v[q];
            }
            wave_lds_order();
            load_x(min(b + waves, n_blk - 1), v);
            w[1 - a].load(row, min(b + waves, n_blk - 1));
            f32x4 sum[TT];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int g = m / PG;
                u32x4 xv[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) xv[t] = mine[(16 * t + (lane & 15)) * 16 + ((4 * m + quarter) ^ (lane & 15))];
                const u32x4 f = Q4Op<E>::decode(w[a].c[m], Q4Op<E>::zero(w[a].zero(g)));
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    sum[t] = Q4Op<E>::mfma(xv[t], f, m % PG == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[t]);
                if ((m + 1) % PG == 0) {
                    const float sc = w[a].scale(g);
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(sc, sum[t][i], acc[t][i]);
                }
            }
        }
    }
    __syncthreads();
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int t = 0; t < TT; ++t) part[(wv * TT + t) * 64 + lane] = acc[t];
    __syncthreads();
    const float *sums = reinterpret_cast<const float *>(lds);
    for (int o = threadIdx.x; o < 16 * n_tok; o += blockDim.x) {
        const int r = o % 16, t = o / 16;
        const int at = (t / 16 * 64 + (t % 16 / 4) * 16 + r) * 4 + t % 4;
        float s = 0.0f;
        for (int k = 0; k < waves; ++k) s += sums[k * TT * 256 + at];
        if (row0 + r < n_rows) q4_store<E>(y, f32, t * ldy + row0 + r, Q4Op<E>::UNIT * (alpha * s), beta);
    }
}

// More tokens: a workgroup's four waves own 16 RT rows each and share a tile of
// 16 TT tokens, a block of 128 columns at a time, through LDS (16-byte pieces
// exchanged within a row by the token's number, so that 16 tokens' pieces lie in
// different banks).  Every fragment of W is decoded once and used TT times; its
// codes go straight to registers, a block ahead.  With few tiles the columns are
// split over workgroups, whose sums k_q4_join adds.  12288 x 12288, bf16, groups of 64,
// zero points, 48 tokens: 32 us, of which 2.6 are the start, 2.9 the stores; the vector
// unit (17 instructions to decode 8 codes) and the matrix cores are busy a third of the
// time each, and codes arrive at 2.6 TB/s.  fp16, groups of 128, 513 tokens: 185 to 190
// us, 816 to 837 TFLOP/s, 432 workgroups on 512 places, vector unit 82 us and matrix
// cores 70, which overlap in part.  TT of 8 with sums in accumulation registers, 16 rows of a wave, and
// codes two blocks ahead were slower.
template <class E, bool ZP, int G, int RT, int TT, bool SPLIT>
__global__ __launch_bounds__(256, 2) void k_q4_tile(int n_rows, int n_cols, int n_blk, int row_tiles, int tok_tiles,
                                                    int split, const char *__restrict__ tiles, int n_tok, float alpha,
                                                    const typename E::T *__restrict__ x, int64_t ldx, float beta,
                                                    void *__restrict__ y, bool f32, int64_t ldy,
                                                    float *__restrict__ parts) {
    constexpr int PG = G / 32, TN = 16 * TT, XA = RT == 4 || TT == 4 ? 1 : 2;
    __shared__ u32x4 xt[2][TN * 16];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), quarter = lane / 16;
    // neighbouring workgroups run on different XCDs; every 8th one shares a row tile, whose codes one L2 then holds
    const int id = blockIdx.x, group = id / (8 * tok_tiles), in = id % (8 * tok_tiles);
    const int wide = min(8, row_tiles - group * 8);
    const int row_tile = group * 8 + in % wide, tok_tile = in / wide;
    const int64_t row0 = ((int64_t)row_tile * 4 + wv) * (16 * RT);
    const int t0 = tok_tile * TN;
    const int b0 = (int)((int64_t)n_blk * blockIdx.y / split), b1 = (int)((int64_t)n_blk * (blockIdx.y + 1) / split);
    Q4Rows<ZP, G> rows[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)                     // tiles past the end: not stored
        rows[r] = Q4Rows<ZP, G>(tiles, min(row0 / 16 + r, (int64_t)(n_rows - 1) / 16), n_blk);
    const int piece = threadIdx.x % 16;
    const typename E::T *xr[TT];
    int slot[TT];
#pragma unroll
    for (int q = 0; q < TT; ++q) {
        const int t = (threadIdx.x + 256 * q) / 16;
        xr[q] = x + (int64_t)min(t0 + t, n_tok - 1) * ldx;
        slot[q] = t * 16 + (piece ^ (t & 15));
    }
    auto load_x = [&](int b, u32x4 (&v)[TT]) {
#pragma unroll
        for (int q = 0; q < TT; ++q) v[q] = q4_token_ahead(xr[q], b * Q4_BLOCK + piece * 8, n_cols);
    };
    auto keep_x = [&](int b, u32x4 *to, u32x4 (&v)[TT]) {
        if (b == n_cols / Q4_BLOCK) {
#pragma unroll
            for (int q = 0; q < TT; ++q) v[q] = q4_token_placed(v[q], b * Q4_BLOCK + piece * 8, n_cols);
        }
#pragma unroll
        for (int q = 0; q < TT; ++q) to[slot[q]] = v[q];
    };
    Q4Piece<E, ZP, G> w[2][RT];
    u32x4 v[XA][TT];                                 // x of the next block, and of the one after it where there is room
    load_x(b0, v[0]);
    if constexpr (XA == 2) load_x(min(b0 + 1, b1 - 1), v[1]);
#pragma unroll
    for (int r = 0; r < RT; ++r) w[0][r].load(rows[r], b0);
    keep_x(b0, xt[0], v[0]);
    f32x4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    for (int bb = b0; bb < b1; bb += 2) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int b = bb + a;
            if (b >= b1) break;
            const u32x4 *now = xt[a];
            // x first: what waits for it does not wait for the codes behind it
            load_x(min(b + XA, b1 - 1), v[XA == 2 ? a : 0]);
#pragma unroll
            for (int r = 0; r < RT; ++r) w[1 - a][r].load(rows[r], min(b + 1, b1 - 1));
            __builtin_amdgcn_sched_barrier(0);
            f32x4 sum[RT][TT];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int g = m / PG;
                u32x4 xv[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) xv[t] = now[(16 * t + (lane & 15)) * 16 + ((4 * m + quarter) ^ (lane & 15))];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const u32x4 f = Q4Op<E>::decode(w[a][r].c[m], Q4Op<E>::zero(w[a][r].zero(g)));
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        sum[r][t] = Q4Op<E>::mfma(xv[t], f, m % PG == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[r][t]);
                }
                if ((m + 1) % PG == 0) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float sc = w[a][r].scale(g);
#pragma unroll
                        for (int t = 0; t < TT; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(sc, sum[r][t][i], acc[r][t][i]);
                    }
                }
                // keeps the fragments of one product in registers at a time
                __builtin_amdgcn_sched_barrier(0);
            }
            keep_x(min(b + 1, b1 - 1), xt[1 - a], v[XA == 2 ? 1 - a : 0]);
            __syncthreads();
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = row0 + 16 * r + (lane & 15);
        if (row >= n_rows) continue;
        // the lane's token of each tile is 16 rows of the result further
        float *part = SPLIT ? parts + ((int64_t)blockIdx.y * n_tok + t0 + 4 * quarter) * n_rows + row : nullptr;
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = t0 + 16 * t + 4 * quarter + i;
                if (tok >= n_tok) continue;
                if constexpr (SPLIT)
                    part[(int64_t)(16 * t + i) * n_rows] = acc[r][t][i];
                else
                    q4_store<E>(y, f32, (int64_t)tok * ldy + row, Q4Op<E>::UNIT * (alpha * acc[r][t][i]), beta);
            }
    }
}

// Adds the parts, in order: 4 results for a thread, 8 parts on their way together
// (5 parts of 48 x 12288, 12 MB from the second-level caches: 4.5 us, half of it the
// launch and one chain of loads).
template <class E>
__global__ __launch_bounds__(256) void k_q4_join(int n_rows, int n_tok, int split, float alpha, float beta,
                                                 const float *__restrict__ parts, void *__restrict__ y, bool f32,
                                                 int64_t ldy) {
    constexpr int U = 8;
    const int64_t n = (int64_t)n_rows * n_tok, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int64_t from = min(i, max((int64_t)0, n - 4));         // the last thread starts early
    if (n < 4) {
        for (int64_t j = i; j < n; ++j) {
            float v = 0.0f;
            for (int k = 0; k < split; ++k) v += parts[k * n + j];
            q4_store<E>(y, f32, j / n_rows * ldy + j % n_rows, Q4Op<E>::UNIT * (alpha * v), beta);
        }
        return;
    }
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < split; k0 += U) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = __builtin_bit_cast(f32x4, load_any<F32, 4>(parts + min(k0 + u, split - 1) * n + from));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < split) sum += v[u];
    }
    int64_t t = from / n_rows;
    int row = (int)(from - t * n_rows);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (from + j >= i) q4_store<E>(y, f32, t * ldy + row, Q4Op<E>::UNIT * (alpha * sum[j]), beta);
        if (++row == n_rows) row = 0, ++t;
    }
}

// y = beta * y where W has no columns.
template <class E>
__global__ __launch_bounds__(256) void k_q4_scale(int n_rows, int64_t n, float beta, void *__restrict__ y, bool f32,
                                                  int64_t ldy) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        q4_store<E>(y, f32, i / n_rows * ldy + i % n_rows, 0.0f, beta);
}

// The records from the rows: a workgroup writes the records of four blocks, a wave
// each.  What lies past the last row is zeros, and so are the scales of groups past the
// last column, whatever the caller's arrays hold there: x is zero in them, and a NaN
// for a scale would come through.  Bound by HBM: 12288 x 12288 in 30 us, 5.2 TB/s.
__global__ __launch_bounds__(256) void k_q4_tiles(int64_t n_rows, int n_cols, int n_blk, int gb, int64_t n_rec,
                                                  int rec_bytes, const u32x4 *__restrict__ codes,
                                                  const unsigned short *__restrict__ scales,
                                                  const unsigned char *__restrict__ zeros, char *__restrict__ tiles) {
    const int lane = __lane_id();
    const int64_t rec = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (rec >= n_rec) return;
    const int64_t tile = rec / n_blk, row = tile * 16 + (lane & 15);
    const int b = (int)(rec - tile * n_blk);
    char *out = tiles + rec * rec_bytes;
    const u32x4 none = {0u, 0u, 0u, 0u};
    reinterpret_cast<u32x4 *>(out)[lane] = row < n_rows ? codes[(row * n_blk + b) * 4 + lane / 16] : none;
    for (int i = lane; i < 16 * gb; i += 64) {
        const int64_t r = tile * 16 + i / gb, at = (r * n_blk + b) * gb + i % gb;
        const bool in = r < n_rows && b * Q4_BLOCK + i % gb * (Q4_BLOCK / gb) < n_cols;
        reinterpret_cast<unsigned short *>(out + Q4_SCALES)[i] = in ? scales[at] : (unsigned short)0;
        if (zeros) reinterpret_cast<unsigned char *>(out + Q4_SCALES + 32 * gb)[i] = r < n_rows ? zeros[at] : (unsigned char)0;
    }
}

// Codes of a dense weight, one thread per group.  Symmetric: s = max |w| / 7,
// q = w / s rounded to even + 8.  With zero points: s = (max(w, 0) - min(w, 0)) / 15,
// z = -min(w, 0) / s and q = w / s + z, each rounded to even and kept in 0 .. 15.
// s is rounded to its type (at most its largest number) before it divides.  Once per
// weight, and as simple as that: a lane reads its group twice, an element at a time, far
// from its neighbours' (12288 x 12288: 0.6 ms from fp16 in groups of 32, 4.7 in groups of
// 128, 5.5 from fp32; its bytes take 0.07 to 0.13).
template <class S, class W>
__global__ __launch_bounds__(256) void k_q4_quantize(int64_t n_groups, int n_cols, int gpr, int group,
                                                     const typename W::T *__restrict__ w, int64_t ldw,
                                                     unsigned *__restrict__ codes, typename S::T *__restrict__ scales,
                                                     unsigned char *__restrict__ zeros) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= n_groups) return;
    const int64_t row = id / gpr;
    const int64_t c0 = (id - row * gpr) * group, c1 = min(c0 + group, (int64_t)n_cols);
    const typename W::T *src = w + row * ldw;
    float lo = 0.0f, hi = 0.0f;
    for (int64_t c = c0; c < c1; ++c) {
        const float v = (float)src[c];
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    const float largest = std::is_same<S, F16>::value ? 65504.0f : 3.3895314e38f;
    // the difference of two large numbers may pass fp32's range; a fifteenth of each does not
    const float want = zeros ? hi / 15.0f - lo / 15.0f : fmaxf(hi, -lo) / 7.0f;
    const typename S::T st = (typename S::T)fminf(want, largest);
    const float s = (float)st;
    const float z = zeros ? (s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f) : 8.0f;
    scales[id] = st;
    if (zeros) zeros[id] = (unsigned char)z;
    unsigned *dst = codes + (row * (gpr * (int64_t)group / Q4_BLOCK)) * Q4_WORDS;
    for (int i = 0; i < group / 8; ++i) {
        const int64_t c = c0 + 8 * i;
        unsigned word = 0;
        for (int e = 0; e < 8; ++e) {
            const float v = c + e < n_cols ? (float)src[c + e] : 0.0f;
            const float q = s > 0.0f ? fminf(fmaxf(rintf(v / s) + z, 0.0f), 15.0f) : z;
            word |= (unsigned)q << (4 * q4_place(e));
        }
        const int in = (int)(c % Q4_BLOCK);
        dst[c / Q4_BLOCK * Q4_WORDS + 4 * (in % 32 / 8) + in / 32] = word;
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int Q4_MAX_COLS = 1 << 30;

spmv_status check_weight(int32_t n_rows, int32_t n_cols, int32_t group, int32_t dtype) {
    if (n_rows < 0 || n_cols < 0) return fail(SPMV_ERR_INVALID_VALUE, "negative size");
    if (n_cols > Q4_MAX_COLS) return fail(SPMV_ERR_UNSUPPORTED, "more than %d columns are not supported", Q4_MAX_COLS);
    if (!q4_group_ok(group)) return fail(SPMV_ERR_INVALID_VALUE, "group must be 32, 64 or 128, not %d", group);
    if (!dtype_ok(dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", dtype);
    if (dtype == SPMV_F32) return fail(SPMV_ERR_UNSUPPORTED, "scales and x are fp16 or bf16");
    return SPMV_OK;
}

template <class F>
spmv_status by_weight(int32_t dtype, bool zp, int32_t group, F f) {
    auto g = [&](auto e, auto z) {
        if (group == 32) return f(e, z, std::integral_constant<int, 32>{});
        if (group == 64) return f(e, z, std::integral_constant<int, 64>{});
        return f(e, z, std::integral_constant<int, 128>{});
    };
    if (dtype == SPMV_F16) return zp ? g(F16{}, std::true_type{}) : g(F16{}, std::false_type{});
    return zp ? g(BF16{}, std::true_type{}) : g(BF16{}, std::false_type{});
}

// How a product of more than QF_TOKENS tokens is cut: rows of a wave, tokens of a tile, parts of the columns.
struct Tiling {
    int rt, tt, row_tiles, tok_tiles, split;
};
constexpr int QT_MIN_BLOCKS = 4;     // blocks of columns of a part at least
Tiling tiling(int64_t n_rows, int64_t n_cols, int64_t n_tok, bool wide) {
    Tiling t;
    t.tt = (int)std::min<int64_t>(4, ceil_div(n_tok, 16));
    // 64 rows of a wave share a fragment of x, where their sums fit the registers: 513
    // tokens of 12288 x 12288 192 us against 230 with 32 rows (fp16, groups of 128).  With
    // zero points 3 (fp16) to 20 registers (bf16) spill: 214 against 227 and 304 against
    // 256, 200 tokens of 4096 x 12288 in fp16 43 against 40; groups of 64 spill 140 and
    // more: 775 to 1160 against 252 to 290; groups of 32 with zero points 1300 against 295
    t.rt = n_tok > 64 && wide ? 4 : 2;
    t.row_tiles = (int)ceil_div(n_rows, 64 * t.rt);
    t.tok_tiles = (int)ceil_div(n_tok, 16 * t.tt);
    // two workgroups on each CU: 48 tokens of 12288 x 12288 (bf16, groups of 64, zero
    // points) 35.9 us with 512 and 38.9 with 768, whose parts take longer to add
    const int64_t tiles = (int64_t)t.row_tiles * t.tok_tiles, groups = 512;
    t.split = (int)std::max<int64_t>(1, std::min(groups / tiles, q4_blocks(n_cols) / QT_MIN_BLOCKS));
    return t;
}
// bytes of LDS of k_q4_few
size_t few_lds(int64_t n_cols, int64_t n_tok, int waves) {
    return std::max<size_t>((size_t)n_tok * (q4_blocks(n_cols) * 16 + 1) * 16, (size_t)waves * 1024);
}
// fewer than 8 columns: what reads x ahead takes 8 of them at least
int few_tokens(int64_t n_cols) { return n_cols < 8 ? 16 : QF_TOKENS; }
bool few(int64_t n_cols, int64_t n_tok) {
    return n_cols < 8 || (n_tok <= QF_TOKENS && few_lds(n_cols, n_tok, 0) <= QF_LDS);
}
// Whether k_q4_mid takes the product: every 16 rows read x again, which costs less
// than a second launch up to 130 to 160 MB (f16, groups of 128: 4096 x 4096, 16
// tokens, 34 MB, 8.0 us against 10.6 by tiles; 64 tokens, 134 MB, 11.6 against 12.1; 4096 x
// 4608, 64 tokens, 151 MB, 12.2 against 14.0; 12288 x 12288, 16 tokens, 302 MB, 29 against
// 20.5).  The bytes do not say all: with 33 tokens and more a CU has one workgroup, and
// where the row tiles leave CUs without one or need a second round the tiles are faster
// from less on (2048 x 8704, 64 tokens, 143 MB, 19.5 against 14.4; 4608 x 4608, 48 tokens,
// 127 MB, 17.6 against 13.5).
constexpr int64_t QM_BYTES = 160000000;
bool mid(int64_t n_rows, int64_t n_cols, int64_t n_tok) {
    return n_tok <= 64 && ceil_div(n_rows, 16) * (ceil_div(n_tok, 16) * 16) * n_cols * 2 <= QM_BYTES;
}
size_t split_bytes(int64_t n_rows, int64_t n_cols, int64_t n_tok) {
    if (n_rows == 0 || n_cols == 0 || few(n_cols, n_tok) || mid(n_rows, n_cols, n_tok)) return 0;
    // the larger of both tilings: the size does not depend on the group
    size_t most = 0;
    for (const bool wide : {false, true}) {
        const Tiling t = tiling(n_rows, n_cols, n_tok, wide);
        if (t.split > 1) most = std::max(most, (size_t)t.split * n_tok * n_rows * 4);
    }
    return most;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status q4_quantize(int32_t n_rows, int32_t n_cols, int32_t group, const void *w, int32_t w_dtype,
                                   int64_t ldw, int32_t dtype, uint32_t *codes, void *scales, uint8_t *zeros,
                                   void *stream) {
    spmv_status st = check_weight(n_rows, n_cols, group, dtype);
    if (st != SPMV_OK) return st;
    if (!dtype_ok(w_dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", w_dtype);
    if (ldw < n_cols) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_rows == 0 || n_cols == 0) return SPMV_OK;
    if (!w || !codes || !scales) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    const int64_t gpr = q4_blocks(n_cols) * (Q4_BLOCK / group), n = gpr * n_rows;
    st = check_grid(ceil_div(n, 256));
    if (st != SPMV_OK) return st;
    auto run = [&](auto s, auto e) {
        typedef decltype(s) S;
        typedef decltype(e) W;
        k_q4_quantize<S, W><<<(int)ceil_div(n, 256), 256, 0, as_stream(stream)>>>(
            n, n_cols, (int)gpr, group, static_cast<const typename W::T *>(w), ldw, codes,
            static_cast<typename S::T *>(scales), zeros);
    };
    auto by_w = [&](auto s) {
        if (w_dtype == SPMV_F16)
            run(s, F16{});
        else if (w_dtype == SPMV_BF16)
            run(s, BF16{});
        else
            run(s, F32{});
    };
    if (dtype == SPMV_F16)
        by_w(F16{});
    else
        by_w(BF16{});
    SPMV_LAUNCHED("k_q4_quantize");
    return SPMV_OK;
}

extern "C" spmv_status q4_tiles_size(int32_t n_rows, int32_t n_cols, int32_t group, int32_t with_zeros, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_weight(n_rows, n_cols, group, SPMV_F16);
    if (st != SPMV_OK) return st;
    *bytes = (size_t)ceil_div(n_rows, 16) * (size_t)q4_blocks(n_cols) * q4_record(group, with_zeros != 0);
    return SPMV_OK;
}

extern "C" spmv_status q4_tiles(int32_t n_rows, int32_t n_cols, int32_t group, const uint32_t *codes,
                                const void *scales, const uint8_t *zeros, void *tiles, size_t tiles_bytes, void *stream) {
    size_t need = 0;
    spmv_status st = q4_tiles_size(n_rows, n_cols, group, zeros != nullptr, &need);
    if (st != SPMV_OK) return st;
    if (need == 0) return SPMV_OK;
    if (!codes || !scales || !tiles) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (tiles_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "tiles of %zu bytes are smaller than %zu", tiles_bytes, need);
    if (!aligned16(codes) || !aligned16(tiles)) return fail(SPMV_ERR_UNSUPPORTED, "codes and tiles must be 16-byte aligned");
    const int64_t n_blk = q4_blocks(n_cols), n_rec = ceil_div(n_rows, 16) * n_blk;
    st = check_grid(ceil_div(n_rec, 4));
    if (st != SPMV_OK) return st;
    k_q4_tiles<<<(int)ceil_div(n_rec, 4), 256, 0, as_stream(stream)>>>(
        n_rows, n_cols, (int)n_blk, Q4_BLOCK / group, n_rec, (int)q4_record(group, zeros != nullptr),
        reinterpret_cast<const u32x4 *>(codes), static_cast<const unsigned short *>(scales), zeros,
        static_cast<char *>(tiles));
    SPMV_LAUNCHED("k_q4_tiles");
    return SPMV_OK;
}

extern "C" spmv_status q4_workspace_size(int32_t n_rows, int32_t n_cols, int32_t n_tok, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    if (n_rows < 0 || n_cols < 0 || n_tok < 0) return fail(SPMV_ERR_INVALID_VALUE, "negative size");
    if (n_cols > Q4_MAX_COLS) return fail(SPMV_ERR_UNSUPPORTED, "more than %d columns are not supported", Q4_MAX_COLS);
    // the most that any batch of up to n_tok tokens needs: full tiles of tokens, as long as there is a split
    size_t most = split_bytes(n_rows, n_cols, n_tok);
    for (int64_t t = QF_TOKENS; t < n_tok; t = t < 16 ? 16 : t < 64 ? t + 16 : t + 64) {
        const size_t b = split_bytes(n_rows, n_cols, t);
        if (b == 0 && t > 64) break;
        most = std::max(most, b);
    }
    *bytes = most;
    return SPMV_OK;
}

extern "C" spmv_status q4_matmul(int32_t n_rows, int32_t n_cols, int32_t group, int32_t with_zeros, const void *tiles,
                                 int32_t dtype, int32_t n_tok, float alpha, const void *x, int64_t ldx, float beta,
                                 void *y, int32_t y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    spmv_status st = check_weight(n_rows, n_cols, group, dtype);
    if (st != SPMV_OK) return st;
    if (n_tok < 0) return fail(SPMV_ERR_INVALID_VALUE, "negative size");
    if (!dtype_ok(y_dtype)) return fail(SPMV_ERR_INVALID_VALUE, "element type %d is not a spmv_dtype", y_dtype);
    if (y_dtype != SPMV_F32 && y_dtype != dtype) return fail(SPMV_ERR_UNSUPPORTED, "y must be fp32 or have x's type");
    if (ldx < n_cols || ldy < n_rows) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_rows == 0 || n_tok == 0) return SPMV_OK;
    if (!y || (n_cols > 0 && (!tiles || !x))) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (!aligned16(tiles)) return fail(SPMV_ERR_UNSUPPORTED, "tiles must be 16-byte aligned");
    hipStream_t s = as_stream(stream);
    const bool f32 = y_dtype == SPMV_F32;
    if (n_cols == 0) {
        const int64_t n = (int64_t)n_rows * n_tok;
        const int grid = (int)std::min<int64_t>(ceil_div(n, 256), 65536);
        if (dtype == SPMV_F16)
            k_q4_scale<F16><<<grid, 256, 0, s>>>(n_rows, n, beta, y, f32, ldy);
        else
            k_q4_scale<BF16><<<grid, 256, 0, s>>>(n_rows, n, beta, y, f32, ldy);
        SPMV_LAUNCHED("k_q4_scale");
        return SPMV_OK;
    }
    const int n_blk = (int)q4_blocks(n_cols);
    st = check_grid(ceil_div(n_rows, 16), 64 * QF_WAVES);
    if (st != SPMV_OK) return st;
    if (few(n_cols, n_tok))
        return by_weight(dtype, with_zeros != 0, group, [&](auto e, auto zp, auto g) -> spmv_status {
            typedef decltype(e) E;
            typedef typename E::T T;
            constexpr bool ZP = decltype(zp)::value;
            constexpr int G = decltype(g)::value;
            const int waves = (int)std::min<int64_t>(QF_WAVES, ceil_div(n_blk, QF_UNROLL));
            auto run = [&](auto tp, int64_t t0, int n) {
                k_q4_few<E, ZP, G, decltype(tp)::value>
                    <<<(int)ceil_div(n_rows, 16), 64 * waves, few_lds(n_cols, n, waves), s>>>(
                        n_rows, n_cols, n_blk, static_cast<const char *>(tiles), n, alpha,
                        static_cast<const T *>(x) + t0 * ldx, ldx, beta,
                        static_cast<char *>(y) + t0 * ldy * dtype_size(y_dtype), f32, ldy);
            };
            if (n_tok == 1)
                run(std::integral_constant<int, 1>{}, 0, 1);
            else                                           // more than one turn only for fewer than 8 columns
                for (int64_t t0 = 0; t0 < n_tok; t0 += few_tokens(n_cols))
                    run(std::integral_constant<int, 16>{}, t0, (int)std::min<int64_t>(n_tok - t0, few_tokens(n_cols)));
            SPMV_LAUNCHED("k_q4_few");
            return SPMV_OK;
        });
    if (mid(n_rows, n_cols, n_tok))
        return by_weight(dtype, with_zeros != 0, group, [&](auto e, auto zp, auto g) -> spmv_status {
            typedef decltype(e) E;
            typedef typename E::T T;
            constexpr bool ZP = decltype(zp)::value;
            constexpr int G = decltype(g)::value;
            const int waves = (int)std::min<int64_t>(QF_WAVES, n_blk);
            auto run = [&](auto tt) {
                constexpr int TT = decltype(tt)::value;
                k_q4_mid<E, ZP, G, TT><<<(int)ceil_div(n_rows, 16), 64 * waves, (size_t)waves * TT * 4096, s>>>(
                    n_rows, n_cols, n_blk, static_cast<const char *>(tiles), n_tok, alpha, static_cast<const T *>(x), ldx,
                    beta, y, f32, ldy);
            };
            if (n_tok <= 16)
                run(std::integral_constant<int, 1>{});
            else if (n_tok <= 32)
                run(std::integral_constant<int, 2>{});
            else if (n_tok <= 48)
                run(std::integral_constant<int, 3>{});
            else
                run(std::integral_constant<int, 4>{});
            SPMV_LAUNCHED("k_q4_mid");
            return SPMV_OK;
        });
    const Tiling t = tiling(n_rows, n_cols, n_tok, group == 128 && !with_zeros);
    const size_t need = split_bytes(n_rows, n_cols, n_tok);
    if (need && !workspace) return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (q4_workspace_size gives its size)");
    if (workspace_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    st = check_grid((int64_t)t.row_tiles * t.tok_tiles);
    if (st != SPMV_OK) return st;
    st = by_weight(dtype, with_zeros != 0, group, [&](auto e, auto zp, auto g) -> spmv_status {
        typedef decltype(e) E;
        typedef typename E::T T;
        constexpr bool ZP = decltype(zp)::value;
        constexpr int G = decltype(g)::value;
        auto launch = [&](auto rt, auto tt, auto split) {
            k_q4_tile<E, ZP, G, decltype(rt)::value, decltype(tt)::value, decltype(split)::value>
                <<<dim3((unsigned)(t.row_tiles * t.tok_tiles), (unsigned)t.split), 256, 0, s>>>(
                    n_rows, n_cols, n_blk, t.row_tiles, t.tok_tiles, t.split, static_cast<const char *>(tiles), n_tok,
                    alpha, static_cast<const T *>(x), ldx, beta, y, f32, ldy, static_cast<float *>(workspace));
        };
        auto run = [&](auto rt, auto tt) {
            t.split > 1 ? launch(rt, tt, std::true_type{}) : launch(rt, tt, std::false_type{});
        };
        const std::integral_constant<int, 2> two;
        const std::integral_constant<int, 4> four;
        if (t.rt == 4) {
            if constexpr (G == 128 && !ZP) run(four, four);
        } else if (t.tt == 4)
            run(two, four);
        else if (t.tt == 3)
            run(two, std::integral_constant<int, 3>{});
        else if (t.tt == 2)
            run(two, two);
        else
            run(two, std::integral_constant<int, 1>{});
        SPMV_LAUNCHED("k_q4_tile");
        return SPMV_OK;
    });
    if (st != SPMV_OK || t.split == 1) return st;
    const int grid = (int)ceil_div((int64_t)n_rows * n_tok, 1024);
    if (dtype == SPMV_F16)
        k_q4_join<F16><<<grid, 256, 0, s>>>(n_rows, n_tok, t.split, alpha, beta, static_cast<const float *>(workspace), y,
                                            f32, ldy);
    else
        k_q4_join<BF16><<<grid, 256, 0, s>>>(n_rows, n_tok, t.split, alpha, beta, static_cast<const float *>(workspace), y,
                                             f32, ldy);
    SPMV_LAUNCHED("k_q4_join");
    return SPMV_OK;
}
