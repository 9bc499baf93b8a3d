// A layer of gated experts with 4-bit weights for the few tokens of a decoding
// step, on gfx950, in two launches:
//   h[t, c] = silu(Wg x[t]) * (Wu x[t]),  y[t] = sum_c w[t, c] Wd h[t, c]
// with the weights of token t's c-th expert.  The bound is reading each used
// expert's weights once.
//
// Up (k_moe_up): a workgroup owns 16 gate rows and the same 16 up rows of one
// expert and finds the expert's tokens among the keys itself: no sort comes
// before it.  Where there are fewer slots than experts the grid counts slots,
// and the first slot of an expert does its work.
// Down (k_moe_down): a workgroup owns 16 rows of y for all experts; its waves
// take an expert (or a part of its columns) each, add the weighted results to
// sums of their own in LDS, and these are added in order at the end: no
// atomics, the same bits on every call.
//
// h is kept as three bf16 numbers whose sum has all of fp32's 24 bits (cut, not
// rounded, so that the largest numbers stay finite): the down product is
// three products of the same fragment, and it is the decoding and the weights'
// bytes that cost.
#include "q4.hpp"

#include <algorithm>

namespace spmv {
namespace {

constexpr int ME_MAX_TOK = 256;
constexpr int ME_MAX_SLOTS = 4096;
constexpr int ME_MAX_EXPERTS = 1024;
constexpr int ME_UNROLL = 4;

// h as three bf16 planes [slot][h_ld]
struct Hidden {
    unsigned short *p;
    int64_t ld, plane;
};

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

template <class E, bool ZP, int G, int U, int RT>
__device__ __forceinline__ void up_products(const Q4Piece<E, ZP, G, U> (&w)[RT], const u32x4 (&x)[U][4], f32x4 (&acc)[RT]) {
    constexpr int GB = Q4_BLOCK / G, PG = G / 32;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int g = 0; g < GB; ++g) {
                const typename Q4Op<E>::Zero nz = Q4Op<E>::zero(w[r].zero(u, g));
                f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int m = g * PG; m < (g + 1) * PG; ++m)
                    sum = Q4Op<E>::mfma(x[u][m], Q4Op<E>::decode(w[r].c[u][m], nz), sum);
                const float s = w[r].scale(u, g) * Q4Op<E>::UNIT;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(s, sum[i], acc[r][i]);
            }
}

template <class E, bool ZP, int G>
__global__ __launch_bounds__(512) void k_moe_up(int n_tok, int top_k, int n_experts, int dim, int inter, int n_blk,
                                                bool by_slot, const int *__restrict__ keys,
                                                const char *__restrict__ tiles,
                                                const typename E::T *__restrict__ x, int64_t ldx, Hidden h) {
    constexpr int U = ME_UNROLL;
    extern __shared__ __attribute__((aligned(16))) f32x4 part[];       // [waves][2][64]
    __shared__ unsigned short list[ME_MAX_TOK];                        // slots of the expert, one per token
    __shared__ int n_list;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    int e = blockIdx.y;
    if (by_slot) {
        const int s = blockIdx.y;
        e = keys[s];
        int before = 0;
        for (int i = threadIdx.x; i < s; i += blockDim.x) before |= keys[i] == e;
        if (__syncthreads_or(before) || (unsigned)e >= (unsigned)n_experts) return;
    }
    if (wv == 0) {
        int n = 0;
        for (int t0 = 0; t0 < n_tok; t0 += 64) {
            const int t = t0 + lane;
            int c = top_k;
            if (t < n_tok)
                for (c = 0; c < top_k && keys[t * top_k + c] != e; ++c) {}
            const unsigned long long has = __ballot(t < n_tok && c < top_k);
            if (t < n_tok && c < top_k) list[n + __popcll(has & ((1ull << lane) - 1))] = (unsigned short)(t * top_k + c);
            n += __popcll(has);
        }
        if (lane == 0) n_list = n;
    }
    __syncthreads();
    const int n = n_list;
    const int row0 = blockIdx.x * 16, quarter = lane / 16;
    Q4Rows<ZP, G> rows[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
        rows[r] = Q4Rows<ZP, G>::any(tiles, ((int64_t)e * 2 + r) * inter + min(row0 + (lane & 15), inter - 1), n_blk);
    const int whole = dim / (Q4_BLOCK * U);
    for (int first = 0; first < n; first += 16) {
        const typename E::T *xr = x + (int64_t)(list[min(first + (lane & 15), n - 1)] / top_k) * ldx;
        f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        for (int p = wv; p < whole; p += waves) {
            const int b = p * U;
            Q4Piece<E, ZP, G, U> w[2];
            u32x4 xv[U][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) w[r].load(rows[r], b);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    xv[u][m] = *reinterpret_cast<const u32x4_any *>(xr + (int64_t)(b + u) * Q4_BLOCK + 32 * m + 8 * quarter);
            up_products<E, ZP, G, U, 2>(w, xv, acc);
        }
        for (int b = whole * U + wv; b < n_blk; b += waves) {
            Q4Piece<E, ZP, G, 1> w[2];
            u32x4 xv[1][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) w[r].load(rows[r], b);
#pragma unroll
            for (int m = 0; m < 4; ++m)
                xv[0][m] = q4_token_piece(xr, (int64_t)b * Q4_BLOCK + 32 * m + 8 * quarter, dim);
            up_products<E, ZP, G, 1, 2>(w, xv, acc);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) part[(wv * 2 + r) * 64 + lane] = acc[r];
        __syncthreads();
        const float *sums = reinterpret_cast<const float *>(part);
        for (int o = threadIdx.x; o < 16 * min(16, n - first); o += blockDim.x) {
            const int row = o % 16, t = o / 16;
            const int at = ((t / 4) * 16 + row) * 4 + t % 4;
            float gate = 0.0f, up = 0.0f;
            for (int w = 0; w < waves; ++w) {
                gate += sums[w * 512 + at];
                up += sums[w * 512 + 256 + at];
            }
            unsigned short v[3] = {0, 0, 0};                            // columns past inter are zeros
            if (row0 + row < inter) split3(gate / (1.0f + expf(-gate)) * up, v);
#pragma unroll
            for (int i = 0; i < 3; ++i) h.p[i * h.plane + list[first + t] * h.ld + row0 + row] = v[i];
        }
        __syncthreads();
    }
}

template <class E, bool ZP, int G>
__global__ __launch_bounds__(1024) void k_moe_down(int n_tok, int top_k, int n_experts, int dim, int n_blk,
                                                   const int *__restrict__ keys, const float *__restrict__ weights,
                                                   const char *__restrict__ tiles, Hidden h,
                                                   void *__restrict__ y, bool f32, int64_t ldy) {
    constexpr int GB = Q4_BLOCK / G, PG = G / 32, U = ME_UNROLL;
    typedef Q4Op<BF16> Op;
    extern __shared__ __attribute__((aligned(16))) float sums[];        // [waves][n_tok][16], then what follows
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
    const int quarter = lane / 16, slots = n_tok * top_k;
    float *mine = sums + (size_t)wv * n_tok * 16;
    int *mark = reinterpret_cast<int *>(sums + (size_t)waves * n_tok * 16);     // first slot of each expert
    float *share = reinterpret_cast<float *>(mark + n_experts) + wv * n_tok;   // the wave's list: weight ..
    short *key = reinterpret_cast<short *>(reinterpret_cast<float *>(mark + n_experts) + waves * n_tok);
    unsigned short *list = reinterpret_cast<unsigned short *>(key + slots) + wv * n_tok;   // .. and slot
    unsigned short *active = reinterpret_cast<unsigned short *>(key + slots) + waves * n_tok;
    __shared__ int n_active;
    for (int i = threadIdx.x; i < n_experts; i += blockDim.x) mark[i] = slots;
    for (int i = threadIdx.x; i < waves * n_tok * 16; i += blockDim.x) sums[i] = 0.0f;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const int e = keys[i];
        const bool in = (unsigned)e < (unsigned)n_experts;
        key[i] = (short)(in ? e : -1);
        if (in) atomicMin(&mark[e], i);
    }
    __syncthreads();
    if (wv == 0) {                                                      // the experts in the order of their first slots
        int n = 0;
        for (int s0 = 0; s0 < slots; s0 += 64) {
            const int s = s0 + lane, e = s < slots ? key[s] : -1;
            const bool first = e >= 0 && mark[e] == s;
            const unsigned long long has = __ballot(first);
            if (first) active[n + __popcll(has & ((1ull << lane) - 1))] = (unsigned short)e;
            n += __popcll(has);
        }
        if (lane == 0) n_active = n;
    }
    __syncthreads();
    const int na = n_active;
    // with fewer experts than waves, several waves share an expert's columns
    const int pieces = (n_blk + U - 1) / U;
    const int split = na > 0 ? min(pieces, max(1, (waves + na - 1) / na)) : 1;
    const int row0 = blockIdx.x * 16;
    for (int unit = wv; unit < na * split; unit += waves) {
        const int e = __builtin_amdgcn_readfirstlane(active[unit / split]), k0 = unit % split;
        int n = 0;
        for (int t0 = 0; t0 < n_tok; t0 += 64) {
            const int t = t0 + lane;
            int slot = -1;
            float w = 0.0f;
            if (t < n_tok)
                for (int c = top_k - 1; c >= 0; --c)                    // an expert chosen twice counts with both weights
                    if (key[t * top_k + c] == e) {
                        slot = t * top_k + c;
                        w += weights ? weights[slot] : 1.0f;
                    }
            const unsigned long long has = __ballot(slot >= 0);
            if (slot >= 0) {
                const int at = n + __popcll(has & ((1ull << lane) - 1));
                list[at] = (unsigned short)slot;
                share[at] = w;
            }
            n += __popcll(has);
        }
        __builtin_amdgcn_wave_barrier();
        const Q4Rows<ZP, G> row = Q4Rows<ZP, G>::any(tiles, (int64_t)e * dim + min(row0 + (lane & 15), dim - 1), n_blk);
        for (int first = 0; first < n; first += 16) {
            const unsigned short *hr = h.p + (int64_t)list[min(first + (lane & 15), n - 1)] * h.ld + 8 * quarter;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
            auto block = [&](const auto &w, int u, int b) {
                u32x4 v[3][4];
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        v[i][m] = *reinterpret_cast<const u32x4 *>(hr + i * h.plane + (int64_t)b * Q4_BLOCK + 32 * m);
#pragma unroll
                for (int g = 0; g < GB; ++g) {
                    const Op::Zero nz = Op::zero(w.zero(u, g));
                    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int m = g * PG; m < (g + 1) * PG; ++m) {
                        const u32x4 f = Op::decode(w.c[u][m], nz);
#pragma unroll
                        for (int i = 2; i >= 0; --i) sum = Op::mfma(v[i][m], f, sum);
                    }
                    const float sc = w.scale(u, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = fmaf(sc, sum[i], acc[i]);
                }
            };
            for (int p = k0; p < pieces; p += split) {
                const int b0 = p * U;
                if (b0 + U <= n_blk) {
                    Q4Piece<E, ZP, G, U> w;
                    w.load(row, b0);
#pragma unroll
                    for (int u = 0; u < U; ++u) block(w, u, b0 + u);
                } else {
                    for (int b = b0; b < n_blk; ++b) {
                        Q4Piece<E, ZP, G, 1> w;
                        w.load(row, b);
                        block(w, 0, b);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = first + quarter * 4 + i;
                if (at < n) {                                           // a token is once in the list: no two lanes meet
                    float *d = mine + (list[at] / top_k) * 16 + (lane & 15);
                    *d = fmaf(share[at], acc[i], *d);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int o = threadIdx.x; o < n_tok * 16; o += blockDim.x) {
        const int row = row0 + o % 16;
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += sums[(size_t)w * n_tok * 16 + o];
        if (row < dim) {
            const int64_t at = (int64_t)(o / 16) * ldy + row;
            if (f32)
                static_cast<float *>(y)[at] = v;
            else
                static_cast<typename E::T *>(y)[at] = (typename E::T)v;
        }
    }
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

size_t down_lds(int waves, int n_tok, int top_k, int n_experts) {
    const size_t slots = (size_t)n_tok * top_k;
    return (size_t)waves * n_tok * (16 * 4 + 4 + 2) + (size_t)n_experts * 4 + slots * 2 +
           std::min<size_t>(slots, n_experts) * 2;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status moe_workspace_size(int32_t n_tok, int32_t top_k, int32_t inter, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_slots(n_tok, top_k, inter);
    if (st != SPMV_OK) return st;
    *bytes = (size_t)n_tok * top_k * hidden_ld(inter) * 3 * 2;
    return SPMV_OK;
}

extern "C" spmv_status moe_apply(int32_t n_tok, int32_t top_k, int32_t n_experts, int32_t dim, int32_t inter,
                                 int32_t group, int32_t with_zeros, const int32_t *keys, const float *weights,
                                 const void *up_tiles, const void *down_tiles, int32_t dtype, const void *x, int64_t ldx, void *y, int32_t y_dtype, int64_t ldy, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    size_t need = 0;
    spmv_status st = moe_workspace_size(n_tok, top_k, inter, &need);
    if (st != SPMV_OK) return st;
    if (n_experts < 1 || dim < 1) return fail(SPMV_ERR_INVALID_VALUE, "n_experts and dim must be >= 1");
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
    const Hidden h = {static_cast<unsigned short *>(workspace), ld, ld * slots};
    const bool by_slot = slots <= n_experts;
    const int up_blk = (int)q4_blocks(dim), down_blk = (int)q4_blocks(inter);
    st = check_grid(ld / 16 * (by_slot ? slots : n_experts), 512);
    if (st != SPMV_OK) return st;
    st = check_grid(ceil_div(dim, 16), 1024);
    if (st != SPMV_OK) return st;
    hipStream_t s = as_stream(stream);
    auto launch = [&](auto e, auto zp, auto g) -> spmv_status {
        typedef decltype(e) E;
        typedef typename E::T T;
        constexpr bool ZP = decltype(zp)::value;
        constexpr int G = decltype(g)::value;
        const int up_waves = (int)std::min<int64_t>(8, ceil_div(up_blk, ME_UNROLL));
        k_moe_up<E, ZP, G><<<dim3((unsigned)(ld / 16), by_slot ? slots : n_experts), 64 * up_waves,
                             (size_t)up_waves * 2048, s>>>(
            n_tok, top_k, n_experts, dim, inter, up_blk, by_slot, keys, static_cast<const char *>(up_tiles),
            static_cast<const T *>(x), ldx, h);
        SPMV_LAUNCHED("k_moe_up");
        // a wave's sums take 64 bytes per token: 16 waves up to 64 tokens, 8 up to 256
        const int waves = n_tok <= 64 ? 16 : 8;
        k_moe_down<E, ZP, G><<<(int)ceil_div(dim, 16), 64 * waves, down_lds(waves, n_tok, top_k, n_experts), s>>>(
            n_tok, top_k, n_experts, dim, down_blk, keys, weights, static_cast<const char *>(down_tiles), h, y,
            y_dtype == SPMV_F32, ldy);
        SPMV_LAUNCHED("k_moe_down");
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
