// A layer of gated experts with 4-bit weights for the few tokens of a decoding
// step, on gfx950, in two launches, or three beyond 64 choices:
//   h[t, c] = silu(Wg x[t]) * (Wu x[t]),  y[t] = sum_c w[t, c] Wd h[t, c]
// with the weights of token t's c-th expert.  The bound is reading each used
// expert's weights once.  Every kernel finds its expert's tokens among the keys
// itself: no sort comes before it.  Where there are fewer choices than experts the
// grid counts choices, and the first choice of an expert does its work.
//
// Up (k_moe_up, k_moe_up_tile): a wave owns 16 gate rows and the same 16 up rows of an
// expert, so that silu and the product are its own registers' work.
// Down, up to 64 choices (k_moe_down): a workgroup owns 16 (or 8) rows of y for all
// experts, and the weighted results are added in LDS, in order.  More (k_moe_down_tile):
// by experts, as the up product, results per choice, which k_moe_sum weights and adds
// by token.  No atomics on results: the same bits on every call.
//
// Measured, and what the weights' bytes take at the rate of a large copy: one token,
// 2 of 8 experts of 2048 x 4096 17 us (26 MB: 5), 9 up and 9 down, each a chain of
// launch, keys, codes and sums; 16 tokens, 8 of 64 of 2048 x 1024 60 us (190 MB: 37),
// 35 + 24 + 5; 200 tokens, 4 of 24 of 4096 x 1500 124 to 142 us (230 MB: 44), 60 + 68 + 6.
//
// h is kept as three bf16 numbers whose sum has all of fp32's 24 bits (cut, not
// rounded, so that the largest numbers stay finite): the down product is
// three products of the same fragment, and it is the decoding and the weights'
// bytes that cost.  It lies in the order in which the down product reads it: an
// expert's tokens (its entries) behind those of smaller experts, 16 at a time, and in
// such a tile of n entries [block][part][8 columns][entry], so that a fragment is
// one run of 64 n bytes.  (With a row per slot, 16 lanes touch 16 cache lines: 125 M
// accesses and 294 us for 200 tokens and 24 experts of 4096 x 1500.)
#include "q4.hpp"

#include <algorithm>

namespace spmv {
namespace {

constexpr int ME_MAX_TOK = 256;
constexpr int ME_MAX_SLOTS = 4096;
constexpr int ME_MAX_EXPERTS = 1024;
constexpr int ME_MAX_WIDTH = 1 << 24;
constexpr int ME_UP_WAVES = 4;
constexpr int ME_FEW_SLOTS = 64;     // choices up to which the down product adds by token itself
constexpr int ME_TURNS = 3;          // workgroups of an expert's rows where its tokens may need several turns
constexpr int ME_DOWN_WAVES = 16;
constexpr int ME_UNROLL = 2;         // blocks of a step of the down product

// Where the tile of entries first .. first + n - 1 of all entries begins, and a
// part of a piece of 8 columns in it (in 16-bit numbers).
__device__ __forceinline__ int64_t hidden_tile(int first, int n_blk) { return (int64_t)first * n_blk * (Q4_BLOCK * 3); }
__device__ __forceinline__ int hidden_piece(int b, int part, int piece, int n) { return ((b * 16 + piece) * 3 + part) * n * 8; }

// v = a + b + c with 8 bits each; an infinity or NaN is whole in the first.
__device__ __forceinline__ void split3(float v, unsigned short (&o)[3]) {
    const unsigned a = __float_as_uint(v) & 0xFFFF0000u;
    const bool finite = (a & 0x7F800000u) != 0x7F800000u;
    // a NaN whose upper bits are those of an infinity stays one
    o[0] = (unsigned short)((v != v ? 0x7FC00000u : a) >> 16);
    const float r = finite ? v - __uint_as_float(a) : 0.0f;
    const unsigned b = __float_as_uint(r) & 0xFFFF0000u;
    o[1] = (unsigned short)(b >> 16);
    o[2] = (unsigned short)(__float_as_uint(r - __uint_as_float(b)) >> 16);
}

// An expert's tokens, found by a workgroup of the up product: list[0 .. n) (each
// token once, ascending), where its entries begin among all, and the room there is
// for them (its choices).
struct Entries {
    int n, base, room;
};
struct EntryLds {
    unsigned short list[ME_MAX_TOK];
    int count[ME_UP_WAVES], below[ME_UP_WAVES], equal[ME_UP_WAVES];
};
static_assert(ME_MAX_TOK <= 64 * ME_UP_WAVES, "a thread looks at one token's choices");
// The expert of this workgroup, or -1 if another one does its work.
__device__ __forceinline__ int expert_of(int n_experts, bool by_slot, const int *__restrict__ keys) {
    if (!by_slot) return blockIdx.y;
    const int s = blockIdx.y, e = keys[s];
    int before = 0;
    for (int i = threadIdx.x; i < s; i += 64 * ME_UP_WAVES) before |= keys[i] == e;
    return __syncthreads_or(before) || (unsigned)e >= (unsigned)n_experts ? -1 : e;
}
__device__ __forceinline__ Entries find_entries(int n_tok, int top_k, int e, const int *__restrict__ keys, EntryLds &l) {
    constexpr int U = 8;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), t = threadIdx.x;
    int lo = 0, eq = 0;
    bool mine = false;
    for (int c0 = 0; c0 < top_k; c0 += U) {
        int k[U];
#pragma unroll
        for (int u = 0; u < U; ++u) k[u] = t < n_tok && c0 + u < top_k ? keys[t * top_k + c0 + u] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo += __popcll(__ballot(k[u] >= 0 && k[u] < e));
            eq += __popcll(__ballot(k[u] == e));
            mine |= k[u] == e;
        }
    }
    const unsigned long long has = __ballot(mine);
    if (lane == 0) l.count[wv] = __popcll(has), l.below[wv] = lo, l.equal[wv] = eq;
    __syncthreads();
    Entries r = {0, 0, 0};
    int at = 0;
#pragma unroll
    for (int w = 0; w < ME_UP_WAVES; ++w) {
        if (w < wv) at += l.count[w];
        r.n += l.count[w], r.base += l.below[w], r.room += l.equal[w];
    }
    if (mine) l.list[at + __popcll(has & ((1ull << lane) - 1))] = (unsigned short)t;
    __syncthreads();
    r.n = __builtin_amdgcn_readfirstlane(r.n);
    r.base = __builtin_amdgcn_readfirstlane(r.base);
    r.room = __builtin_amdgcn_readfirstlane(r.room);
    return r;
}

// Where the results of this expert's choices will be: place[slot] = entry.
__device__ __forceinline__ void store_places(int top_k, int e, const Entries &en, const EntryLds &l,
                                             const int *__restrict__ keys, int *__restrict__ place) {
    for (int i = threadIdx.x; i < en.n; i += 64 * ME_UP_WAVES)
        for (int s = l.list[i] * top_k, c = 0; c < top_k; ++c, ++s)
            if (keys[s] == e) place[s] = en.base + i;
}

// One block's products of gate and up rows with TT tiles of x, as they lie in LDS.
template <class E, bool ZP, int G, int TT>
__device__ __forceinline__ void up_block(const Q4Piece<E, ZP, G> (&w)[2], const u32x4 *xt, f32x4 (&acc)[2][TT]) {
    constexpr int PG = G / 32;
    const int lane = __lane_id(), quarter = lane / 16;
    f32x4 sum[2][TT];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int g = m / PG;
        u32x4 xv[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) xv[t] = xt[(16 * t + (lane & 15)) * 16 + ((4 * m + quarter) ^ (lane & 15))];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const u32x4 f = Q4Op<E>::decode(w[r].c[m], Q4Op<E>::zero(w[r].zero(g)));
#pragma unroll
            for (int t = 0; t < TT; ++t)
                sum[r][t] = Q4Op<E>::mfma(xv[t], f, m % PG == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[r][t]);
        }
        if ((m + 1) % PG == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float sc = w[r].scale(g);
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(sc, sum[r][t][i], acc[r][t][i]);
            }
        }
    }
}

// h of the 16 columns from row0 on and the 16 entries from `first` on, of which `here` are there.
template <class E>
__device__ __forceinline__ void store_hidden(const f32x4 &gate, const f32x4 &up, const Entries &en, int first, int here,
                                             int row0, int inter, int h_blk, unsigned short *__restrict__ h) {
    const int lane = __lane_id(), row = row0 + (lane & 15), in = min(16, en.room - first);
    if (row >= h_blk * Q4_BLOCK) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 4 * (lane / 16) + i;
        if (at >= here) continue;
        unsigned short o[3] = {0, 0, 0};                                // columns past inter are zeros
        if (row < inter) {
            const float g = Q4Op<E>::UNIT * gate[i], u = Q4Op<E>::UNIT * up[i];
            split3(g / (1.0f + expf(-g)) * u, o);
        }
        unsigned short *d = h + hidden_tile(en.base + first, h_blk) + at * 8 + row % 8;
#pragma unroll
        for (int k = 0; k < 3; ++k) d[hidden_piece(row / Q4_BLOCK, k, row % Q4_BLOCK / 8, in)] = o[k];
    }
}

// Few tokens of an expert: a wave brings its block of x into LDS of its own and
// takes every parts-th block of its rows, so that no wave waits for another before the
// sums at the end (a row of x per lane, straight to registers, is 64 cache accesses for
// a load).  16 tokens, 8 of 64 experts, zero points: 127 MB of weights in 35 us, 3.6 TB/s;
// the vector unit is busy a quarter of the time, waiting for codes the rest.
template <class E, bool ZP, int G>
__global__ __launch_bounds__(64 * ME_UP_WAVES, 4) void k_moe_up(int n_tok, int top_k, int n_experts, int dim, int inter,
                                                                int n_blk, int h_blk, int parts, bool by_slot,
                                                                const int *__restrict__ keys,
                                                                const char *__restrict__ tiles,
                                                                const typename E::T *__restrict__ x, int64_t ldx,
                                                                unsigned short *__restrict__ h, int *__restrict__ place) {
    __shared__ u32x4 xt[ME_UP_WAVES][16 * 16];                         // a wave's block of x, then its sums
    __shared__ EntryLds el;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), quarter = lane / 16;
    const int e = __builtin_amdgcn_readfirstlane(expert_of(n_experts, by_slot, keys));
    if (e < 0) return;
    const int part = wv % parts, row0 = ((int)blockIdx.x * (ME_UP_WAVES / parts) + wv / parts) * 16;
    Q4Rows<ZP, G> rows[2];
    Q4Piece<E, ZP, G> w[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        rows[r] = Q4Rows<ZP, G>::any(tiles, ((int64_t)e * 2 + r) * inter + min(row0 + (lane & 15), inter - 1), n_blk);
        w[0][r].load(rows[r], min(part, n_blk - 1));                    // on its way while the tokens are found
    }
    const Entries en = find_entries(n_tok, top_k, e, keys, el);
    if (en.n == 0) return;
    if (place && blockIdx.x == 0) store_places(top_k, e, en, el, keys, place);
    u32x4 *mine = xt[wv];
    const int piece = lane % 16;
    for (int first = 0; first < en.n; first += 16) {
        const int here = min(16, en.n - first);
        const typename E::T *xr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) xr[q] = x + (int64_t)el.list[min(first + 4 * q + quarter, en.n - 1)] * ldx;
        auto load_x = [&](int b, u32x4 (&v)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = q4_token_ahead(xr[q], b * Q4_BLOCK + piece * 8, dim);
        };
        f32x4 acc[2][1] = {{{0.0f, 0.0f, 0.0f, 0.0f}}, {{0.0f, 0.0f, 0.0f, 0.0f}}};
        u32x4 v[4];
        load_x(min(part, n_blk - 1), v);
        if (first > 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) w[0][r].load(rows[r], min(part, n_blk - 1));
        }
        for (int bb = part; bb < n_blk; bb += 2 * parts) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int b = bb + a * parts;
                if (b >= n_blk) break;
                if (b == dim / Q4_BLOCK) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = q4_token_placed(v[q], b * Q4_BLOCK + piece * 8, dim);
                }
                wave_lds_order();                                      // after the reads of the block before
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int t = 4 * q + quarter;
                    mine[t * 16 + (piece ^ t)] = v[q];
                }
                wave_lds_order();
                load_x(min(b + parts, n_blk - 1), v);
#pragma unroll
                for (int r = 0; r < 2; ++r) w[1 - a][r].load(rows[r], min(b + parts, n_blk - 1));
                up_block<E, ZP, G, 1>(w[a], mine, acc);
            }
        }
        f32x4 *sums = reinterpret_cast<f32x4 *>(mine);                 // [2][64] of the wave's 4 KB
        wave_lds_order();
#pragma unroll
        for (int r = 0; r < 2; ++r) sums[r * 64 + lane] = acc[r][0];
        __syncthreads();
        if (part == 0) {                                               // the wave of the first columns adds the others'
            f32x4 gate = acc[0][0], up = acc[1][0];
            for (int p = 1; p < parts; ++p) {
                const f32x4 *other = reinterpret_cast<const f32x4 *>(xt[wv + p]);
                gate += other[lane];
                up += other[64 + lane];
            }
            store_hidden<E>(gate, up, en, first, here, row0, inter, h_blk, h);
        }
        __syncthreads();
    }
}

// More: the waves of a workgroup share the block of x of 16 TT tokens, and a fragment
// of W is decoded once for all of them.  Experts with more tokens than that have their
// turns in workgroups of their own, up to ME_TURNS (200 tokens over 24 uneven experts,
// up to 3 turns: 60 us; 77 when one workgroup takes them all).  With groups of 128 and
// no zero points three workgroups fit a CU if one block of codes is on its way, not two:
// 60 us against 75.  Decoding is a third of the vector unit's time there; the rest is
// waiting, at 2.5 TB/s of weights.
template <class E, bool ZP, int G, int TT>
__global__ __launch_bounds__(64 * ME_UP_WAVES, TT <= 3 && G == 128 && !ZP ? 3 : 2) void k_moe_up_tile(int n_tok, int top_k, int n_experts, int dim,
                                                                     int inter, int n_blk, int h_blk,
                                                                     const int *__restrict__ keys,
                                                                     const char *__restrict__ tiles,
                                                                     const typename E::T *__restrict__ x, int64_t ldx,
                                                                     unsigned short *__restrict__ h, int *__restrict__ place) {
    // blocks of codes on their way: one where three workgroups fit a CU with it, and where
    // scales and zero points of 32 columns leave no registers for two
    constexpr bool THREE = TT <= 3 && G == 128 && !ZP;
    constexpr int TN = 16 * TT, A = THREE || (TT == 3 && G == 32 && ZP) ? 1 : 2;
    __shared__ u32x4 xt[2][TN * 16];
    __shared__ EntryLds el;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int e = blockIdx.y, row0 = ((int)blockIdx.x * ME_UP_WAVES + wv) * 16;
    const Entries en = find_entries(n_tok, top_k, e, keys, el);
    if (place && blockIdx.x == 0 && blockIdx.z == 0) store_places(top_k, e, en, el, keys, place);
    Q4Rows<ZP, G> rows[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
        rows[r] = Q4Rows<ZP, G>::any(tiles, ((int64_t)e * 2 + r) * inter + min(row0 + (lane & 15), inter - 1), n_blk);
    const int piece = threadIdx.x % 16, mine = threadIdx.x / 16;       // this thread's pieces: of entries mine + 16 q
    for (int first = blockIdx.z * TN; first < en.n; first += TN * gridDim.z) {
        const int here = min(TN, en.n - first);
        const typename E::T *xr[TT];
#pragma unroll
        for (int q = 0; q < TT; ++q) xr[q] = x + (int64_t)el.list[min(first + 16 * q + mine, en.n - 1)] * ldx;
        auto load_x = [&](int b, u32x4 (&v)[TT]) {
#pragma unroll
            for (int q = 0; q < TT; ++q) v[q] = q4_token_ahead(xr[q], b * Q4_BLOCK + piece * 8, dim);
        };
        auto keep_x = [&](int b, u32x4 *to, u32x4 (&v)[TT]) {
            if (b == dim / Q4_BLOCK) {
#pragma unroll
                for (int q = 0; q < TT; ++q) v[q] = q4_token_placed(v[q], b * Q4_BLOCK + piece * 8, dim);
            }
#pragma unroll
            for (int q = 0; q < TT; ++q) to[(16 * q + mine) * 16 + (piece ^ mine)] = v[q];
        };
        f32x4 acc[2][TT];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        Q4Piece<E, ZP, G> w[A + 1][2];
        u32x4 v[TT];
        load_x(0, v);
#pragma unroll
        for (int a = 0; a < A; ++a)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[a][r].load(rows[r], min(a, n_blk - 1));
        keep_x(0, xt[0], v);
        __syncthreads();
        for (int bb = 0; bb < n_blk; bb += A + 1) {
#pragma unroll
            for (int a = 0; a <= A; ++a) {
                const int b = bb + a;
                if (b >= n_blk) break;
                load_x(min(b + 1, n_blk - 1), v);                      // x first: what waits for it does not wait for the codes
#pragma unroll
                for (int r = 0; r < 2; ++r) w[(a + A) % (A + 1)][r].load(rows[r], min(b + A, n_blk - 1));
                __builtin_amdgcn_sched_barrier(0);
                up_block<E, ZP, G, TT>(w[a], xt[b & 1], acc);
                keep_x(min(b + 1, n_blk - 1), xt[1 - (b & 1)], v);
                __syncthreads();
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (16 * t < here)
                store_hidden<E>(acc[0][t], acc[1][t], en, first + 16 * t, min(16, here - 16 * t), row0, inter, h_blk, h);
    }
}

// Up to 64 choices: a lane holds one, and everything about an expert is ballots over
// them, without a barrier before the sums at the end (found in LDS by all waves: 12 us
// against 9 for one token and 2 experts).  A unit of work is an expert, or a part of its
// columns: 16 waves have one each.
template <class E, bool ZP, int G>
__global__ __launch_bounds__(64 * ME_DOWN_WAVES) void k_moe_down(int n_tok, int top_k, int n_experts, int dim, int rows,
                                                                 int n_blk, const int *__restrict__ keys,
                                                                 const float *__restrict__ weights,
                                                                 const char *__restrict__ tiles,
                                                                 const unsigned short *__restrict__ h,
                                                                 void *__restrict__ y, bool f32, int64_t ldy) {
    constexpr int GB = Q4_BLOCK / G, PG = G / 32, U = ME_UNROLL, W = ME_DOWN_WAVES;
    typedef Q4Op<BF16> Op;
    typedef unsigned long long u64;
    extern __shared__ __attribute__((aligned(16))) float sums[];        // [W][n_tok][16]
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), quarter = lane / 16;
    const int slots = n_tok * top_k;
    const int key = lane < slots ? keys[lane] : -1;
    const float weight = weights && lane < slots ? weights[lane] : 1.0f;
    float *mine = sums + wv * n_tok * 16;
    for (int i = lane; i < n_tok * 16; i += 64) mine[i] = 0.0f;
    wave_lds_order();
    const bool valid = (unsigned)key < (unsigned)n_experts;
    const u64 below = (1ull << lane) - 1;
    const int tok0 = lane / top_k * top_k;                              // first choice of this lane's token
    // first choices of an expert
    u64 firsts = 0, left = __ballot(valid);
    while (left) {
        const int j = __ffsll(left) - 1;
        firsts |= 1ull << j;
        left &= ~__ballot(valid && key == __builtin_amdgcn_readlane(key, j));
    }
    const int na = __popcll(firsts);
    // a unit of work for about every wave: an expert, or a part of its columns.
    // A wave goes through its units' steps (U blocks of 16 entries), the next step's codes on their way.
    const int pieces = (n_blk + U - 1) / U;
    const int split = na > 0 ? min(pieces, (W + na - 1) / na) : 1;
    const int row0 = blockIdx.x * rows, r = lane & (rows - 1), units = na * split;
    struct Step {
        int unit, e, n, base, room, first, k0, p;
        u64 same, lead;
    };
    auto begin = [&](int unit) {
        Step s = {unit, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        if (unit < units) {
            const int a = unit / split;
            u64 m = firsts;
            for (int i = 0; i < a; ++i) m &= m - 1;
            s.k0 = s.p = unit - a * split;
            s.e = __builtin_amdgcn_readlane(key, __ffsll(m) - 1);
            s.same = __ballot(valid && key == s.e);
            // one entry for each token, at its first choice of the expert
            s.lead = __ballot(valid && key == s.e && !(s.same & below & ~((1ull << tok0) - 1)));
            s.n = __popcll(s.lead);
            s.room = __popcll(s.same);
            s.base = __popcll(__ballot(valid && key < s.e));
        }
        return s;
    };
    auto after = [&](Step s) {
        s.p += split;
        if (s.p < pieces) return s;
        s.p = s.k0;
        s.first += 16;
        return s.first < s.n ? s : begin(s.unit + W);
    };
    Q4Piece<E, ZP, G> w[2][U];
    auto load = [&](const Step &s, Q4Piece<E, ZP, G> (&to)[U]) {
        const Q4Rows<ZP, G> row = Q4Rows<ZP, G>::any(tiles, (int64_t)s.e * dim + min(row0 + r, dim - 1), n_blk);
#pragma unroll
        for (int u = 0; u < U; ++u) to[u].load(row, min(s.p * U + u, n_blk - 1));
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    Step s = begin(wv);
    if (s.unit < units) load(s, w[0]);
    while (s.unit < units) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            if (s.unit >= units) break;
            const Step next = after(s);
            load(next.unit < units ? next : s, w[1 - a]);               // always, for the waits behind it
            // up to 5 entries lie with all their parts in one operand of 16 (row part * in + entry)
            const int in = min(16, s.room - s.first);
            const bool packed = in <= 5;
            const u32x4 *ht = reinterpret_cast<const u32x4 *>(h + hidden_tile(s.base + s.first, n_blk));
            const int hl = quarter * 3 * in + min(lane & 15, (packed ? 3 * in : in) - 1);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = s.p * U + u;
                if (b >= n_blk) continue;
                u32x4 v[3][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) v[0][m] = (ht + hidden_piece(b, 0, 4 * m, in) / 8)[hl];
                if (!packed) {
#pragma unroll
                    for (int i = 1; i < 3; ++i)
#pragma unroll
                        for (int m = 0; m < 4; ++m) v[i][m] = (ht + hidden_piece(b, i, 4 * m, in) / 8)[hl];
                }
#pragma unroll
                for (int g = 0; g < GB; ++g) {
                    const Op::Zero nz = Op::zero(w[a][u].zero(g));
                    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int m = g * PG; m < (g + 1) * PG; ++m) {
                        const u32x4 f = Op::decode(w[a][u].c[m], nz);
                        if (!packed) {
                            sum = Op::mfma(v[2][m], f, sum);
                            sum = Op::mfma(v[1][m], f, sum);
                        }
                        sum = Op::mfma(v[0][m], f, sum);
                    }
                    const float sc = w[a][u].scale(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = fmaf(sc, sum[i], acc[i]);
                }
            }
            if (next.unit != s.unit || next.first != s.first) {
                // row i of the result, for all quarters
                auto result = [&](int i) {
                    const float x = (i & 2) ? ((i & 1) ? acc[3] : acc[2]) : ((i & 1) ? acc[1] : acc[0]);
                    return __shfl(x, i / 4 * 16 + (lane & 15));
                };
                for (u64 left = s.same; left; left &= left - 1) {       // an expert chosen twice counts with both weights
                    const int j = __ffsll(left) - 1;
                    const int entry = __popcll(s.lead & ((2ull << j) - 1)) - 1 - s.first;
                    if (entry < 0 || entry >= 16) continue;
                    const float wj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
                    float x = result(entry);
                    if (packed) x = (result(2 * in + entry) + result(in + entry)) + x;
                    float *d = mine + j / top_k * 16 + r;
                    if (lane < rows) *d = fmaf(wj, x, *d);
                }
                acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            s = next;
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < n_tok * rows; o += 64 * W) {
        const int in = o % rows, t = o / rows, row = row0 + in;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += sums[(k * n_tok + t) * 16 + in];
        v *= Op::UNIT;
        if (row < dim) {
            const int64_t at = (int64_t)t * ldy + row;
            if (f32)
                static_cast<float *>(y)[at] = v;
            else
                static_cast<typename E::T *>(y)[at] = (typename E::T)v;
        }
    }
}

// More choices: an expert's rows of W times its entries, 32 rows for a wave, 1 / UNIT of
// them into z [entries][dim]; k_moe_sum weights and adds them by token.  The waves of a
// workgroup share the block of h of 16 TT entries, which lies in memory as it is
// read.  Up to 5 entries lie with all their parts in one operand of 16 (3 n rows of
// it, added at the end).  Three tiles take half a block at a time and fixed places in
// LDS: with whole blocks and places that depend on the entries the addresses do not fit
// the registers (200 tokens, 24 experts of 4096 x 1500: 68 us against 89, turns in
// workgroups of their own included; the matrix instructions alone take 14).
// Bound by waits between barriers, at 1.2 TB/s of weights.
template <class E, bool ZP, int G, int TT>
__global__ __launch_bounds__(64 * ME_UP_WAVES, 2) void k_moe_down_tile(int n_tok, int top_k, int n_experts, int dim,
                                                                       int n_blk, bool by_slot,
                                                                       const int *__restrict__ keys,
                                                                       const char *__restrict__ tiles,
                                                                       const unsigned short *__restrict__ h,
                                                                       float *__restrict__ z) {
    // SEG segments of a block, one at a time: SP pieces of 16 bytes of an entry
    constexpr int SEG = TT == 3 ? 2 : 1, SP = 48 / SEG, SM = 4 / SEG;
    constexpr int RT = 2, PG = G / 32, THREADS = 64 * ME_UP_WAVES, Q = (SP * 16 * TT + THREADS - 1) / THREADS;
    typedef Q4Op<BF16> Op;
    __shared__ u32x4 ht[2][SP * 16 * TT];
    __shared__ EntryLds el;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), quarter = lane / 16;
    const int e = __builtin_amdgcn_readfirstlane(expert_of(n_experts, by_slot, keys));
    if (e < 0) return;
    const int row0 = ((int)blockIdx.x * ME_UP_WAVES + wv) * 16 * RT;
    Q4Rows<ZP, G> rows[RT];
    Q4Piece<E, ZP, G> w[2][RT];
    auto load_first = [&]() {
#pragma unroll
        for (int r = 0; r < RT; ++r) w[0][r].load(rows[r], 0);
    };
#pragma unroll
    for (int r = 0; r < RT; ++r)
        rows[r] = Q4Rows<ZP, G>::any(tiles, (int64_t)e * dim + min(row0 + 16 * r + (lane & 15), dim - 1), n_blk);
    if (blockIdx.z == 0) load_first();                                  // on their way while the entries are found
    const Entries en = find_entries(n_tok, top_k, e, keys, el);
    for (int first = blockIdx.z * 16 * TT; first < en.n; first += 16 * TT * gridDim.z) {
        // the pieces of this turn's tiles: a segment of a tile of n entries is SP n of them in a row
        int n_of[TT], from[TT + 1];
        from[0] = 0;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            n_of[t] = first + 16 * t < en.n ? min(16, en.room - first - 16 * t) : 0;
            from[t + 1] = from[t] + SP * n_of[t];
        }
        // in LDS 48 places for the 8 columns of a tile's entries: 16 part + entry, or, packed,
        // n part + entry; what is not written there reaches rows that are not used
        const bool packed = from[TT] <= SP * 5;
        const u32x4 *src[Q];
        int step[Q], dst[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = min((int)threadIdx.x + THREADS * q, from[TT] - 1);       // past the end: the last one again
            int t = 0;
#pragma unroll
            for (int k = 1; k < TT; ++k) t += c >= from[k];
            int n = n_of[0], f = from[0];
#pragma unroll
            for (int k = 1; k < TT; ++k)
                if (t == k) n = n_of[k], f = from[k];
            src[q] = reinterpret_cast<const u32x4 *>(h + hidden_tile(en.base + first + 16 * t, n_blk)) + (c - f);
            step[q] = SP * n;
            const int place = (c - f) / n, piece = place / 3;
            dst[q] = (t * 4 * SM + piece) * 48 + (place - 3 * piece) * (packed ? n : 16) + (c - f) - place * n;
        }
        auto load_h = [&](int seg, u32x4 (&v)[Q]) {
#pragma unroll
            for (int q = 0; q < Q; ++q) v[q] = src[q][(int64_t)seg * step[q]];
        };
        auto keep_h = [&](u32x4 *to, const u32x4 (&v)[Q]) {
#pragma unroll
            for (int q = 0; q < Q; ++q) to[dst[q]] = v[q];
        };
        f32x4 acc[RT][TT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 v[Q];
        load_h(0, v);
        if (first > 0) load_first();
        keep_h(ht[0], v);
        __syncthreads();
        // NT tiles, or (0) one whose parts lie in one operand: without branches inside
        auto products = [&](auto nt) {
            constexpr int NT = decltype(nt)::value, N = NT ? NT : 1;
            for (int bb = 0; bb < n_blk; bb += 2) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int b = bb + a;
                    if (b >= n_blk) break;
                    f32x4 sum[RT][N];
#pragma unroll
                    for (int seg = 0; seg < SEG; ++seg) {
                        load_h(min(SEG * b + seg + 1, SEG * n_blk - 1), v);   // h first: what waits for it does not wait for the codes
                        if (seg == 0) {
#pragma unroll
                            for (int r = 0; r < RT; ++r) w[1 - a][r].load(rows[r], min(b + 1, n_blk - 1));
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        const int at = SEG == 2 ? seg : a;
                        const u32x4 *now = ht[at] + quarter * 48 + (lane & 15);
#pragma unroll
                        for (int m = SM * seg; m < SM * seg + SM; ++m) {
                            const int g = m / PG, p = 4 * (m - SM * seg) * 48;
                            u32x4 f[RT];
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                f[r] = Op::decode(w[a][r].c[m], Op::zero(w[a][r].zero(g)));
                                if (m % PG == 0) {
#pragma unroll
                                    for (int t = 0; t < N; ++t) sum[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                                }
                            }
                            if constexpr (NT == 0) {
                                const u32x4 x = now[p];
#pragma unroll
                                for (int r = 0; r < RT; ++r) sum[r][0] = Op::mfma(x, f[r], sum[r][0]);
                            } else {
#pragma unroll
                                for (int t = 0; t < N; ++t)
#pragma unroll
                                    for (int i = 2; i >= 0; --i) {
                                        const u32x4 x = now[t * 4 * SM * 48 + p + 16 * i];
#pragma unroll
                                        for (int r = 0; r < RT; ++r) sum[r][t] = Op::mfma(x, f[r], sum[r][t]);
                                    }
                            }
                            if ((m + 1) % PG == 0) {
#pragma unroll
                                for (int r = 0; r < RT; ++r) {
                                    const float sc = w[a][r].scale(g);
#pragma unroll
                                    for (int t = 0; t < N; ++t)
#pragma unroll
                                        for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(sc, sum[r][t][i], acc[r][t][i]);
                                }
                            }
                            // keeps the fragments of one product in registers at a time
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        keep_h(ht[1 - at], v);
                        __syncthreads();
                    }
                }
            }
        };
        if (packed)
            products(std::integral_constant<int, 0>{});
        else if (TT == 1 || n_of[TT > 1 ? 1 : 0] == 0)
            products(std::integral_constant<int, 1>{});
        else if (TT == 2 || n_of[TT - 1] == 0)
            products(std::integral_constant<int, TT < 2 ? TT : 2>{});
        else
            products(std::integral_constant<int, TT>{});
        float *zt = z + (int64_t)(en.base + first) * dim;
        if (packed) {
            // row i of the operand, column col: lane 16 (i / 4) + col, i % 4
            f32x4 *mine = reinterpret_cast<f32x4 *>(ht[0]) + wv * 64;
            const float *s = reinterpret_cast<const float *>(mine);
            const int n = n_of[0];
            auto part = [&](int i, int col) { return s[((i / 4) * 16 + col) * 4 + i % 4]; };
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                wave_lds_order();                                      // after the reads of the rows before
                mine[lane] = acc[r][0];
                wave_lds_order();
                for (int o = lane; o < 16 * (en.n - first); o += 64) {
                    const int i = o / 16, col = o % 16;
                    if (row0 + 16 * r + col < dim)
                        zt[(int64_t)i * dim + row0 + 16 * r + col] = (part(2 * n + i, col) + part(n + i, col)) + part(i, col);
                }
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = row0 + 16 * r + (lane & 15);
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 16 * t + 4 * quarter + i;
                        if (row < dim && first + k < en.n) zt[(int64_t)k * dim + row] = acc[r][t][i];
                    }
            }
        }
    }
}

// y[t] = UNIT * sum over c (ascending) of weights[t, c] * z[place[t, c]]; a lane holds one
// of 64 choices, and the rows of 8 choices are on their way together (800 rows of 4096:
// 13 MB in 5.7 us, most of it the launch and one chain of loads).
template <class E>
__global__ __launch_bounds__(256) void k_moe_sum(int n_tok, int top_k, int n_experts, int dim, int pieces,
                                                 const int *__restrict__ keys, const float *__restrict__ weights,
                                                 const int *__restrict__ place, const float *__restrict__ z,
                                                 void *__restrict__ y, bool f32, int64_t ldy) {
    constexpr int U = 8;
    const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int lane = __lane_id(), t = (int)(id / pieces), col = (int)(id - (int64_t)t * pieces) * 64 + lane;
    if (t >= n_tok) return;
    const float *zc = z + min(col, dim - 1);
    float v = 0.0f;
    for (int c0 = 0; c0 < top_k; c0 += 64) {
        const int s = t * top_k + min(c0 + lane, top_k - 1);
        const bool in = c0 + lane < top_k && (unsigned)keys[s] < (unsigned)n_experts;
        const int at = place[s];                                        // of a dropped choice: not used
        const float w = weights ? weights[s] : 1.0f;
        unsigned long long left = __ballot(in);
        while (left) {
            float x[U], f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = left ? __ffsll(left) - 1 : -1;
                left &= left - 1;
                f[u] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j & 63));
                x[u] = j >= 0 ? zc[(int64_t)__builtin_amdgcn_readlane(at, j & 63) * dim] : 0.0f;
                if (j < 0) f[u] = 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) v = fmaf(f[u], x[u], v);
        }
    }
    if (col >= dim) return;
    v *= Q4Op<BF16>::UNIT;
    if (f32)
        static_cast<float *>(y)[t * ldy + col] = v;
    else
        static_cast<typename E::T *>(y)[t * ldy + col] = (typename E::T)v;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
spmv_status check_slots(int32_t n_tok, int32_t top_k, int32_t inter) {
    if (n_tok < 0 || top_k < 1 || inter < 1) return fail(SPMV_ERR_INVALID_VALUE, "n_tok must be >= 0, top_k and inter >= 1");
    if (n_tok > ME_MAX_TOK) return fail(SPMV_ERR_UNSUPPORTED, "more than %d tokens are not supported", ME_MAX_TOK);
    if ((int64_t)n_tok * top_k > ME_MAX_SLOTS)
        return fail(SPMV_ERR_UNSUPPORTED, "more than %d choices of an expert are not supported", ME_MAX_SLOTS);
    return SPMV_OK;
}
int64_t hidden_ld(int32_t inter) { return q4_blocks(inter) * Q4_BLOCK; }

// The workspace's parts: h; beyond ME_FEW_SLOTS choices also z and every choice's place in it.
struct Parts {
    size_t z, place, total;
};
Parts parts_of(int64_t n_tok, int64_t top_k, int64_t dim, int64_t inter) {
    const size_t slots = (size_t)(n_tok * top_k);
    Parts p = {slots * (size_t)hidden_ld((int32_t)inter) * 6, 0, 0};
    p.total = p.z;
    if (slots > ME_FEW_SLOTS) {
        p.place = p.z + slots * (size_t)dim * 4;
        p.total = p.place + slots * 4;
    }
    return p;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status moe_workspace_size(int32_t n_tok, int32_t top_k, int32_t dim, int32_t inter, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_slots(n_tok, top_k, inter);
    if (st != SPMV_OK) return st;
    if (dim < 1) return fail(SPMV_ERR_INVALID_VALUE, "dim must be >= 1");
    const Parts p = parts_of(n_tok, top_k, dim, inter);
    *bytes = p.total;
    return SPMV_OK;
}

extern "C" spmv_status moe_apply(int32_t n_tok, int32_t top_k, int32_t n_experts, int32_t dim, int32_t inter,
                                 int32_t group, int32_t with_zeros, const int32_t *keys, const float *weights,
                                 const void *up_tiles, const void *down_tiles, int32_t dtype, const void *x,
                                 int64_t ldx, void *y, int32_t y_dtype, int64_t ldy, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    size_t need = 0;
    spmv_status st = moe_workspace_size(n_tok, top_k, dim, inter, &need);
    if (st != SPMV_OK) return st;
    if (n_experts < 1) return fail(SPMV_ERR_INVALID_VALUE, "n_experts must be >= 1");
    if (dim < 8) return fail(SPMV_ERR_UNSUPPORTED, "layers of a width below 8 are not supported");
    if (dim > ME_MAX_WIDTH || inter > ME_MAX_WIDTH)
        return fail(SPMV_ERR_UNSUPPORTED, "widths above %d are not supported", ME_MAX_WIDTH);
    if (n_experts > ME_MAX_EXPERTS) return fail(SPMV_ERR_UNSUPPORTED, "more than %d experts are not supported", ME_MAX_EXPERTS);
    if (!q4_group_ok(group)) return fail(SPMV_ERR_INVALID_VALUE, "group must be 32, 64 or 128, not %d", group);
    if (!dtype_ok(dtype) || !dtype_ok(y_dtype)) return fail(SPMV_ERR_INVALID_VALUE, "an element type is not a spmv_dtype");
    if (dtype == SPMV_F32) return fail(SPMV_ERR_UNSUPPORTED, "scales and x are fp16 or bf16");
    if (y_dtype != SPMV_F32 && y_dtype != dtype) return fail(SPMV_ERR_UNSUPPORTED, "y must be fp32 or have x's type");
    if (ldx < dim || ldy < dim) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_tok == 0) return SPMV_OK;
    if (!keys || !up_tiles || !down_tiles || !x || !y)
        return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    if (!aligned16(up_tiles) || !aligned16(down_tiles)) return fail(SPMV_ERR_UNSUPPORTED, "tiles must be 16-byte aligned");
    if (!workspace) return fail(SPMV_ERR_INVALID_VALUE, "workspace is NULL (moe_workspace_size gives its size)");
    if (workspace_bytes < need)
        return fail(SPMV_ERR_INVALID_VALUE, "workspace of %zu bytes is smaller than %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SPMV_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
    const int slots = n_tok * top_k;
    const int64_t ld = hidden_ld(inter);
    const bool by_slot = slots <= n_experts;
    const int up_blk = (int)q4_blocks(dim), down_blk = (int)q4_blocks(inter);
    // parts of the columns in the up product: enough waves for the card
    const int64_t groups = by_slot ? slots : n_experts, up_row_tiles = ld / 16 * groups;
    // tokens of an expert by their number if the choices are even
    const bool tile_up = slots > 12 * groups;
    int parts = 1;
    while (!tile_up && parts < ME_UP_WAVES && parts < up_blk && up_row_tiles * parts < 4096) parts *= 2;
    const int64_t up_grid = ceil_div(ld / 16, ME_UP_WAVES / parts);
    st = check_grid(up_grid * groups * ME_TURNS, 64 * ME_UP_WAVES);
    if (st != SPMV_OK) return st;
    // 8 rows for a workgroup of the down product where 16 would leave compute units without one
    const int rows = ceil_div(dim, 16) < 256 ? 8 : 16;
    st = check_grid(ceil_div(dim, rows), 64 * ME_DOWN_WAVES);
    if (st != SPMV_OK) return st;
    const Parts p = parts_of(n_tok, top_k, dim, inter);
    const bool tile_down = slots > ME_FEW_SLOTS;
    const int64_t down_grid = ceil_div(dim, 32 * ME_UP_WAVES), pieces = ceil_div(dim, 64);
    st = check_grid(down_grid * groups * ME_TURNS, 64 * ME_UP_WAVES);
    if (st != SPMV_OK) return st;
    float *z = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.z);
    int *place = tile_down ? reinterpret_cast<int *>(static_cast<char *>(workspace) + p.place) : nullptr;
    hipStream_t s = as_stream(stream);
    unsigned short *h = static_cast<unsigned short *>(workspace);
    auto launch = [&](auto e, auto zp, auto g) -> spmv_status {
        typedef decltype(e) E;
        typedef typename E::T T;
        constexpr bool ZP = decltype(zp)::value;
        constexpr int G = decltype(g)::value;
        auto turns = [&](int tt) { return (unsigned)std::min<int64_t>(ME_TURNS, ceil_div(n_tok, 16 * tt)); };
        auto up = [&](auto tt) {
            constexpr int TT = decltype(tt)::value;
            k_moe_up_tile<E, ZP, G, TT>
                <<<dim3((unsigned)up_grid, (unsigned)groups, turns(TT)), 64 * ME_UP_WAVES, 0, s>>>(
                    n_tok, top_k, n_experts, dim, inter, up_blk, down_blk, keys, static_cast<const char *>(up_tiles),
                    static_cast<const T *>(x), ldx, h, place);
        };
        if (!tile_up)
            k_moe_up<E, ZP, G><<<dim3((unsigned)up_grid, (unsigned)groups), 64 * ME_UP_WAVES, 0, s>>>(
                n_tok, top_k, n_experts, dim, inter, up_blk, down_blk, parts, by_slot, keys,
                static_cast<const char *>(up_tiles), static_cast<const T *>(x), ldx, h, place);
        else if (slots <= 24 * groups)
            up(std::integral_constant<int, 2>{});
        else if (slots <= 40 * groups)
            up(std::integral_constant<int, 3>{});
        else if constexpr (G == 128 && !ZP)
            up(std::integral_constant<int, 4>{});
        else                                               // more need more registers than there are
            up(std::integral_constant<int, 3>{});
        SPMV_LAUNCHED("k_moe_up");
        if (!tile_down) {
            k_moe_down<E, ZP, G><<<(int)ceil_div(dim, rows), 64 * ME_DOWN_WAVES, (size_t)ME_DOWN_WAVES * n_tok * 64, s>>>(
                n_tok, top_k, n_experts, dim, rows, down_blk, keys, weights, static_cast<const char *>(down_tiles), h, y,
                y_dtype == SPMV_F32, ldy);
            SPMV_LAUNCHED("k_moe_down");
            return SPMV_OK;
        }
        auto down = [&](auto tt) {
            constexpr int TT = decltype(tt)::value;
            k_moe_down_tile<E, ZP, G, TT>
                <<<dim3((unsigned)down_grid, (unsigned)groups, turns(TT)), 64 * ME_UP_WAVES, 0, s>>>(
                    n_tok, top_k, n_experts, dim, down_blk, by_slot, keys, static_cast<const char *>(down_tiles), h, z);
        };
        if (slots <= 12 * groups)
            down(std::integral_constant<int, 1>{});
        else if (slots <= 24 * groups)
            down(std::integral_constant<int, 2>{});
        else if constexpr (G == 128 && !ZP)
            down(std::integral_constant<int, 3>{});
        else
            down(std::integral_constant<int, 2>{});
        SPMV_LAUNCHED("k_moe_down_tile");
        k_moe_sum<E><<<(int)ceil_div(n_tok * pieces, 4), 256, 0, s>>>(n_tok, top_k, n_experts, dim, (int)pieces, keys,
                                                                   weights, place, z, y, y_dtype == SPMV_F32, ldy);
        SPMV_LAUNCHED("k_moe_sum");
        return SPMV_OK;
    };
    auto by_group = [&](auto e, auto z) {
        if (group == 32) return launch(e, z, std::integral_constant<int, 32>{});
        if (group == 64) return launch(e, z, std::integral_constant<int, 64>{});
        return launch(e, z, std::integral_constant<int, 128>{});
    };
    if (dtype == SPMV_F16) return with_zeros ? by_group(F16{}, std::true_type{}) : by_group(F16{}, std::false_type{});
    return with_zeros ? by_group(BF16{}, std::true_type{}) : by_group(BF16{}, std::false_type{});
}
