// MACKO products with many tokens on gfx950: y[t, :] = alpha * W x[t, :] + beta * y[t, :],
// for one pruned weight, or for one weight per group of sorted tokens.
//
// With one token the product is a gather (macko.hip).  With more, every
// decoded entry serves all tokens, so a piece of W is decoded into a dense
// fp16 tile in LDS and multiplied with the matrix cores.  A wave owns 16 rows
// and walks slabs of 256 columns: it clears its own 16 x 256 tile, decodes
// into it, and runs eight 16x16x32 products per 16 tokens on it, so waves
// never wait for each other; the waves of a workgroup take turns over the
// slabs of the same rows and add their sums at the end, in order.
//
// A row's columns are known only after everything before them is decoded, so
// a plan built once per weight (macko_spmm_plan) keeps, for each row and slab,
// the 8-entry unit that holds the first entry at or past the slab's start and
// the column before that unit: 4 bytes per 256 columns, 1.3 % of a half
// pruned row.  Eight lanes share a row in the decoding: lane l takes unit
// u0 + l, the gaps are summed in the lane and scanned over the 8 lanes.
// Entries of a unit that belong to a neighbouring slab land in a spare column.
//
// A pruned position multiplies by zero, as in the dense product: an infinity
// or NaN in a token makes that token's outputs NaN and leaves the others alone.
#include "elem.hpp"

#include <algorithm>
#include <type_traits>

namespace spmv {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int SM_SLAB = 256;            // columns of a slab
constexpr int SM_LDW = SM_SLAB + 8;     // halfs per tile row: the spare columns also spread rows over the banks
constexpr int SM_ROWS = 16;
constexpr int SM_UNIT_BITS = 18;        // plan word: unit in the row, and how far back its predecessor's column lies
constexpr int SM_MAX_COLS = 1 << 20;    // (n_cols + 1024) / 8 units fit SM_UNIT_BITS

__device__ __forceinline__ f16x2 as_h2(unsigned int w) { return __builtin_bit_cast(f16x2, w); }

template <int BD>
struct Codes {
    typedef typename std::conditional<BD == 8, u32x2, unsigned int>::type lane_t;
    // the 8 codes of unit u (a word shared with 4 / BD - 1 neighbours for BD < 4)
    static __device__ __forceinline__ lane_t load(const unsigned int *__restrict__ codes, int64_t u) {
        if constexpr (BD == 8)
            return reinterpret_cast<const u32x2 *>(codes)[u];
        else
            return codes[(u * BD) >> 2];
    }
    // inclusive prefix of (code + 1) over the unit's entries
    static __device__ __forceinline__ void prefix(lane_t w, int64_t u, int (&p)[8]) {
        int run = 0;
        if constexpr (BD == 8) {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                run += (int)(((t < 4 ? w.x : w.y) >> (8 * (t & 3))) & 255u) + 1;
                p[t] = run;
            }
        } else {
            const unsigned int ws = BD < 4 ? w >> ((8 * BD * (unsigned)u) & 31u) : w;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                run += (int)((ws >> (BD * t)) & ((1u << BD) - 1u)) + 1;
                p[t] = run;
            }
        }
    }
};

// the unit's 8 values: 16 bytes of fp16 or 8 bytes of int8
template <bool I8>
using vals_t = typename std::conditional<I8, u32x2, u32x4>::type;

// Values t, t + 1 (t even) as the bits of two fp16; int8 exactly, as 1024 + (q + 128) - 1152.
template <bool I8>
__device__ __forceinline__ unsigned int value_pair(const vals_t<I8> &v, int t) {
    if constexpr (!I8) {
        return v[t >> 1];
    } else {
        const unsigned int w = v[t >> 2] ^ 0x80808080u;
        return __builtin_bit_cast(
            unsigned int, as_h2(__builtin_amdgcn_perm(0x64646464u, w, (t & 2) ? 0x04030402u : 0x04010400u)) -
                              f16x2{(_Float16)1152.0f, (_Float16)1152.0f});
    }
}

// Inclusive sum over groups of 8 lanes: within pairs, within quads, then the
// lower quad's total onto the upper quad.  odd, high: all ones in the odd
// lanes, and in the lanes whose bit 1 is set.
constexpr int DPP_QUAD_0022 = 0xA0;
constexpr int DPP_QUAD_1111 = 0x55;
constexpr int DPP_QUAD_3333 = 0xFF;
constexpr int DPP_ROW_SHL4 = 0x104;
__device__ __forceinline__ int scan8(int v, int odd, int high) {
    v += __builtin_amdgcn_update_dpp(0, v, DPP_QUAD_0022, 0xf, 0xf, false) & odd;
    v += __builtin_amdgcn_update_dpp(0, v, DPP_QUAD_1111, 0xf, 0xf, false) & high;
    const int quad = __builtin_amdgcn_update_dpp(0, v, DPP_QUAD_3333, 0xf, 0xf, false);
    return v + __builtin_amdgcn_update_dpp(0, quad, DPP_ROW_SHR4, 0xf, 0xa, false);
}
// The last lane's value of each group of 8.
__device__ __forceinline__ int last8(int v) {
    const int quad = __builtin_amdgcn_update_dpp(0, v, DPP_QUAD_3333, 0xf, 0xf, false);
    return __builtin_amdgcn_update_dpp(quad, quad, DPP_ROW_SHL4, 0xf, 0x5, false);
}

// Plan: one wave per row walks the row's units 64 at a time.
template <int BD>
__global__ __launch_bounds__(256) void k_macko_spmm_plan(int n_rows, int n_slabs, const int *__restrict__ mrp,
                                                         const unsigned int *__restrict__ codes,
                                                         unsigned int *__restrict__ plan) {
    const int lane = __lane_id();
    const int row = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (row >= n_rows) return;
    unsigned int *out = plan + (int64_t)row * (n_slabs + 1);
    const int u0 = mrp[row] / 8, n = (mrp[row + 1] - mrp[row]) / 8;
    int carry = -1;
    for (int b = 0; b < n; b += 64) {
        const bool in = b + lane < n;
        int p[8];
        Codes<BD>::prefix(in ? Codes<BD>::load(codes, (int64_t)u0 + b + lane) : typename Codes<BD>::lane_t{},
                          (int64_t)u0 + b + lane, p);
        const int tot = in ? p[7] : 0;
        const int incl = wave_inclusive_scan(tot);
        const int before = carry + incl - tot;
        carry += __builtin_amdgcn_readlane(incl, 63);
        // slabs whose start lies in (before, before + tot]
        if (in)
            for (int k = (before + SM_SLAB) / SM_SLAB; k <= n_slabs && k * SM_SLAB <= before + tot; ++k)
                out[k] = (unsigned)(b + lane) | ((unsigned)(k * SM_SLAB - 1 - before) << SM_UNIT_BITS);
    }
    for (int k = (carry + SM_SLAB) / SM_SLAB + lane; k <= n_slabs; k += 64) out[k] = (unsigned)n;
}

// x rows copied into 16-byte aligned rows of a multiple of 8 columns.
__global__ __launch_bounds__(256) void k_macko_spmm_pack(int n_tok, int n_cols, int ldp,
                                                         const unsigned short *__restrict__ x, int64_t ldx,
                                                         unsigned short *__restrict__ out) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= ldp) return;
    for (int t = blockIdx.y; t < n_tok; t += gridDim.y)
        out[(int64_t)t * ldp + c] = c < n_cols ? x[(int64_t)t * ldx + c] : (unsigned short)0;
}

struct SpmmArg {
    int n_rows, n_cols, n_slabs, n_tok;
    const int *mrp;
    const unsigned int *codes;
    const void *vals;
    const float *row_scale;
    const unsigned int *plan;
    const int *tok_offsets;
    const unsigned short *x;
    int64_t ldx;
    void *y;
    int64_t ldy;
    float alpha, beta;
    int y_f32, vec_y;
};

// Decodes the slab `k` of the 16 rows from `row0` on into the wave's tile.
template <int BD, bool I8>
__device__ __forceinline__ void decode_slab(const SpmmArg &a, int64_t row0, int rows, int k, int lane,
                                            unsigned short *tile) {
    typedef vals_t<I8> V;
    const int odd = lane & 1 ? -1 : 0, high = lane & 2 ? -1 : 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = 8 * half + (lane >> 3), l = lane & 7;
        int u = 0, end = 0, carry = 0;
        int64_t base = 0;
        if (r < rows) {
            const unsigned int *p = a.plan + (row0 + r) * (a.n_slabs + 1) + k;
            const unsigned int p0 = p[0], p1 = p[1];
            const int m0 = a.mrp[row0 + r], m1 = a.mrp[row0 + r + 1];
            base = m0 / 8;
            u = (int)(p0 & ((1u << SM_UNIT_BITS) - 1u));
            end = min((int)(p1 & ((1u << SM_UNIT_BITS) - 1u)) + 1, (m1 - m0) / 8);
            carry = -1 - (int)(p0 >> SM_UNIT_BITS);      // relative to the slab's first column
        }
        unsigned short *dst = tile + r * SM_LDW;
        for (; __any(u < end); u += 8) {
            const bool in = u + l < end;
            typename Codes<BD>::lane_t w = {};
            V v = {};
            if (in) {
                w = Codes<BD>::load(a.codes, base + u + l);
                v = reinterpret_cast<const V *>(a.vals)[base + u + l];
            }
            int p[8];
            Codes<BD>::prefix(w, base + u + l, p);
            const int tot = in ? p[7] : 0;
            const int incl = scan8(tot, odd, high);
            const int before = carry + incl - tot;
            carry += last8(incl);
            if (in) {
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    const unsigned int h = value_pair<I8>(v, t);
                    dst[min((unsigned)(before + p[t]), (unsigned)SM_SLAB)] = (unsigned short)h;
                    dst[min((unsigned)(before + p[t + 1]), (unsigned)SM_SLAB)] = (unsigned short)(h >> 16);
                }
            }
        }
    }
}

__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Workgroup: rows 16 blockIdx.y .. of group blockIdx.z, tokens 16 NT blockIdx.x ..
// of that group, slabs wave, wave + WAVES, ...
template <int BD, bool I8, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_macko_spmm(SpmmArg a) {
    extern __shared__ __attribute__((aligned(16))) unsigned short lds[];
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int t0 = 0, t1 = a.n_tok;
    if (a.tok_offsets) {
        t0 = min(max(a.tok_offsets[blockIdx.z], 0), a.n_tok);
        t1 = min(max(a.tok_offsets[blockIdx.z + 1], t0), a.n_tok);
    }
    t0 += blockIdx.x * 16 * NT;
    if (t0 >= t1) return;
    const int live = min(NT, (t1 - t0 + 15) / 16);      // token tiles in use
    const int r0 = blockIdx.y * SM_ROWS;
    const int rows = min(SM_ROWS, a.n_rows - r0);
    const int64_t row0 = (int64_t)blockIdx.z * a.n_rows + r0;
    unsigned short *tile = lds + wv * SM_ROWS * SM_LDW;
    const unsigned short *xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = a.x + (int64_t)min(t0 + 16 * i + n, t1 - 1) * a.ldx + 16 * q;
    f32x4 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int k = wv; k < a.n_slabs; k += WAVES) {
        for (int i = lane; i < SM_ROWS * SM_LDW / 8; i += 64)
            *reinterpret_cast<u32x4 *>(tile + 8 * i) = u32x4{0u, 0u, 0u, 0u};
        wave_lds_order();
        decode_slab<BD, I8>(a, row0, rows, k, lane, tile);
        wave_lds_order();
        const int c0 = k * SM_SLAB;
#pragma unroll
        for (int s = 0; s < SM_SLAB; s += 64) {
            if (c0 + s >= a.n_cols) break;              // uniform
            const u32x4 w0 = *reinterpret_cast<const u32x4 *>(tile + n * SM_LDW + s + 16 * q);
            const u32x4 w1 = *reinterpret_cast<const u32x4 *>(tile + n * SM_LDW + s + 16 * q + 8);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (i < live) {                          // uniform
                    // columns past the last are zeros, not what follows the row of x
                    const int c = c0 + s + 16 * q;
                    u32x4 x0 = {0u, 0u, 0u, 0u}, x1 = {0u, 0u, 0u, 0u};
                    if (c < a.n_cols) x0 = *reinterpret_cast<const u32x4 *>(xr[i] + c0 + s);
                    if (c + 8 < a.n_cols) x1 = *reinterpret_cast<const u32x4 *>(xr[i] + c0 + s + 8);
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w0), __builtin_bit_cast(h8, x0),
                                                                    acc[i], 0, 0, 0);
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w1), __builtin_bit_cast(h8, x1),
                                                                    acc[i], 0, 0, 0);
                }
            }
        }
        wave_lds_order();
    }
    // the waves' sums, added in wave order; the tile is free now
    float *sums = reinterpret_cast<float *>(lds);        // [WAVES][NT][64] of f32x4
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(sums + ((wv * NT + i) * 64 + lane) * 4) = acc[i];
    __syncthreads();
    for (int i = wv; i < live; i += WAVES) {
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int w = 0; w < WAVES; ++w) v += *reinterpret_cast<const f32x4 *>(sums + ((w * NT + i) * 64 + lane) * 4);
        const int tok = t0 + 16 * i + n, r = r0 + 4 * q;   // D: row 4 q + j, column (token) n
        if (tok >= t1) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= I8 && r + j < a.n_rows ? a.alpha * a.row_scale[row0 + 4 * q + j] : a.alpha;
        if (a.y_f32) {
            float *y = static_cast<float *>(a.y) + (int64_t)tok * a.ldy + r;
            if (a.vec_y && r + 3 < a.n_rows) {
                if (a.beta != 0.0f) {
                    const f32x4 o = *reinterpret_cast<const f32x4 *>(y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = fmaf(a.beta, o[j], v[j]);
                }
                *reinterpret_cast<f32x4 *>(y) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + j < a.n_rows) y[j] = a.beta != 0.0f ? fmaf(a.beta, y[j], v[j]) : v[j];
            }
        } else {
            _Float16 *y = static_cast<_Float16 *>(a.y) + (int64_t)tok * a.ldy + r;
            if (a.vec_y && r + 3 < a.n_rows) {
                Vec<F16, 4> o;
                if (a.beta != 0.0f) {
                    o = load_vec<F16, 4>(y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = fmaf(a.beta, (float)o.v[j], v[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o.v[j] = (_Float16)v[j];
                store_vec<F16, 4>(y, o);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + j < a.n_rows) y[j] = (_Float16)(a.beta != 0.0f ? fmaf(a.beta, (float)y[j], v[j]) : v[j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool width_ok(int32_t b) { return b == 1 || b == 2 || b == 4 || b == 8; }

spmv_status check_size(int64_t n_rows, int64_t n_cols) {
    if (n_rows < 0 || n_cols < 0) return fail(SPMV_ERR_INVALID_VALUE, "negative size");
    if (n_cols > SM_MAX_COLS) return fail(SPMV_ERR_UNSUPPORTED, "more than %d columns are not supported", SM_MAX_COLS);
    return SPMV_OK;
}

template <int BD, bool I8, int NT, int WAVES>
void launch(const SpmmArg &a, dim3 grid, hipStream_t st) {
    const size_t lds = std::max<size_t>((size_t)WAVES * SM_ROWS * SM_LDW * 2, (size_t)WAVES * NT * 64 * 16);
    k_macko_spmm<BD, I8, NT, WAVES><<<grid, 64 * WAVES, lds, st>>>(a);
}

template <int BD, bool I8>
spmv_status launch_shape(const SpmmArg &a, int n_groups, hipStream_t st) {
    // token tiles per workgroup; groups share n_tok among them, so any of them may have all
    const int nt = n_groups > 1 || a.n_tok > 32 ? 4 : a.n_tok > 16 ? 2 : 1;
    const dim3 grid((unsigned)ceil_div(a.n_tok, 16 * nt), (unsigned)ceil_div(a.n_rows, SM_ROWS), n_groups);
    if (nt == 1)
        launch<BD, I8, 1, 4>(a, grid, st);
    else if (nt == 2)
        launch<BD, I8, 2, 4>(a, grid, st);
    else
        launch<BD, I8, 4, 4>(a, grid, st);
    SPMV_LAUNCHED("k_macko_spmm");
    return SPMV_OK;
}

template <bool I8>
spmv_status spmm_apply(int32_t n_groups, int32_t n_rows, int32_t n_cols, int32_t bdelta, const int32_t *mrow_ptr,
                       const uint32_t *codes, const void *vals, const float *row_scale, const void *plan,
                       const int32_t *tok_offsets, int32_t n_tok, float alpha, const uint16_t *x, int64_t ldx,
                       float beta, void *y, int32_t y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (n_groups < 1 || n_tok < 0) return fail(SPMV_ERR_INVALID_VALUE, "n_groups must be >= 1 and n_tok >= 0");
    spmv_status st = check_size(n_rows, n_cols);
    if (st != SPMV_OK) return st;
    if (!width_ok(bdelta)) return fail(SPMV_ERR_INVALID_VALUE, "code width %d is not 1, 2, 4 or 8", bdelta);
    if (y_dtype != SPMV_F32 && y_dtype != SPMV_F16)
        return fail(dtype_ok(y_dtype) ? SPMV_ERR_UNSUPPORTED : SPMV_ERR_INVALID_VALUE, "y must be fp32 or fp16");
    if (n_groups > 65535 || ceil_div(n_rows, SM_ROWS) > 65535)
        return fail(SPMV_ERR_UNSUPPORTED, "more than 65535 groups or %d rows are not supported", 65535 * SM_ROWS);
    if ((int64_t)n_groups * n_rows > INT32_MAX) return fail(SPMV_ERR_OVERFLOW, "n_groups * n_rows does not fit int32");
    if (ldx < n_cols || ldy < n_rows) return fail(SPMV_ERR_INVALID_VALUE, "a row stride is shorter than the row");
    if (n_groups > 1 && !tok_offsets) return fail(SPMV_ERR_INVALID_VALUE, "tok_offsets is NULL with several groups");
    if (n_rows == 0 || n_tok == 0) return SPMV_OK;
    if (n_cols == 0) return fail(SPMV_ERR_INVALID_VALUE, "n_cols must be positive when there are rows");
    if (!mrow_ptr || !codes || !vals || !plan || !x || !y || (I8 && !row_scale))
        return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    const uintptr_t va = reinterpret_cast<uintptr_t>(vals), ca = reinterpret_cast<uintptr_t>(codes);
    if ((va & (I8 ? 7u : 15u)) || (ca & (bdelta == 8 ? 7u : 3u)))
        return fail(SPMV_ERR_UNSUPPORTED, I8 ? "q must be 8-byte aligned and codes %d-byte aligned"
                                             : "mvals must be 16-byte aligned and codes %d-byte aligned",
                    bdelta == 8 ? 8 : 4);
    hipStream_t s = as_stream(stream);
    SpmmArg a = {n_rows, n_cols, (int)ceil_div(n_cols, SM_SLAB), n_tok, mrow_ptr, codes, vals, row_scale,
                 static_cast<const unsigned int *>(plan), tok_offsets, x, ldx, y, ldy, alpha, beta, y_dtype == SPMV_F32, 0};
    const size_t ysize = dtype_size(y_dtype);
    a.vec_y = ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * ysize - 1)) == 0;
    if (!aligned16(x) || ldx % 8 != 0 || n_cols % 8 != 0) {
        size_t need = 0;
        macko_spmm_workspace_size(n_tok, n_cols, &need);
        if (!workspace || workspace_bytes < need || !aligned16(workspace))
            return fail(SPMV_ERR_INVALID_VALUE,
                        "rows of x that are not 16-byte aligned, or n_cols not a multiple of 8, need a 16-byte aligned "
                        "workspace of %zu bytes", need);
        const int ldp = (int)(ceil_div(n_cols, 8) * 8);
        k_macko_spmm_pack<<<dim3((unsigned)ceil_div(ldp, 256), (unsigned)std::min(n_tok, 65535)), 256, 0, s>>>(
            n_tok, n_cols, ldp, x, ldx, static_cast<unsigned short *>(workspace));
        SPMV_LAUNCHED("k_macko_spmm_pack");
        a.x = static_cast<const unsigned short *>(workspace);
        a.ldx = ldp;
        a.n_cols = ldp;
    }
    switch (bdelta) {
        case 1: return launch_shape<1, I8>(a, n_groups, s);
        case 2: return launch_shape<2, I8>(a, n_groups, s);
        case 4: return launch_shape<4, I8>(a, n_groups, s);
        default: return launch_shape<8, I8>(a, n_groups, s);
    }
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status macko_spmm_plan_size(int32_t n_rows, int32_t n_cols, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    const spmv_status st = check_size(n_rows, n_cols);
    if (st != SPMV_OK) return st;
    *bytes = (size_t)n_rows * (size_t)(ceil_div(n_cols, SM_SLAB) + 1) * 4;
    return SPMV_OK;
}

extern "C" spmv_status macko_spmm_plan(int32_t n_rows, int32_t n_cols, int32_t bdelta, const int32_t *mrow_ptr,
                                       const uint32_t *codes, void *plan, size_t plan_bytes, void *stream) {
    const spmv_status st = check_size(n_rows, n_cols);
    if (st != SPMV_OK) return st;
    if (!width_ok(bdelta)) return fail(SPMV_ERR_INVALID_VALUE, "code width %d is not 1, 2, 4 or 8", bdelta);
    if (n_rows == 0) return SPMV_OK;
    if (n_cols == 0) return fail(SPMV_ERR_INVALID_VALUE, "n_cols must be positive when there are rows");
    if (!mrow_ptr || !codes || !plan) return fail(SPMV_ERR_INVALID_VALUE, "NULL pointer");
    size_t need = 0;
    macko_spmm_plan_size(n_rows, n_cols, &need);
    if (plan_bytes < need) return fail(SPMV_ERR_INVALID_VALUE, "plan of %zu bytes is smaller than %zu", plan_bytes, need);
    if ((reinterpret_cast<uintptr_t>(plan) & 3u) || (reinterpret_cast<uintptr_t>(codes) & (bdelta == 8 ? 7u : 3u)))
        return fail(SPMV_ERR_UNSUPPORTED, "plan must be 4-byte and codes %d-byte aligned", bdelta == 8 ? 8 : 4);
    const int n_slabs = (int)ceil_div(n_cols, SM_SLAB), grid = (int)ceil_div(n_rows, 4);
    hipStream_t s = as_stream(stream);
    unsigned int *p = static_cast<unsigned int *>(plan);
    switch (bdelta) {
        case 1: k_macko_spmm_plan<1><<<grid, 256, 0, s>>>(n_rows, n_slabs, mrow_ptr, codes, p); break;
        case 2: k_macko_spmm_plan<2><<<grid, 256, 0, s>>>(n_rows, n_slabs, mrow_ptr, codes, p); break;
        case 4: k_macko_spmm_plan<4><<<grid, 256, 0, s>>>(n_rows, n_slabs, mrow_ptr, codes, p); break;
        default: k_macko_spmm_plan<8><<<grid, 256, 0, s>>>(n_rows, n_slabs, mrow_ptr, codes, p); break;
    }
    SPMV_LAUNCHED("k_macko_spmm_plan");
    return SPMV_OK;
}

extern "C" spmv_status macko_spmm_workspace_size(int32_t n_tok, int32_t n_cols, size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    if (n_tok < 0) return fail(SPMV_ERR_INVALID_VALUE, "n_tok < 0");
    const spmv_status st = check_size(0, n_cols);
    if (st != SPMV_OK) return st;
    *bytes = (size_t)n_tok * (size_t)(ceil_div(n_cols, 8) * 8) * 2;
    return SPMV_OK;
}

extern "C" spmv_status macko_spmm(int32_t n_groups, int32_t n_rows, int32_t n_cols, int32_t bdelta,
                                  const int32_t *mrow_ptr, const uint32_t *codes, const uint16_t *mvals,
                                  const void *plan, const int32_t *tok_offsets, int32_t n_tok, float alpha,
                                  const uint16_t *x_f16, int64_t ldx, float beta, void *y, int32_t y_dtype, int64_t ldy,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    return spmm_apply<false>(n_groups, n_rows, n_cols, bdelta, mrow_ptr, codes, mvals, nullptr, plan, tok_offsets, n_tok,
                             alpha, x_f16, ldx, beta, y, y_dtype, ldy, workspace, workspace_bytes, stream);
}

extern "C" spmv_status macko_spmm_i8(int32_t n_groups, int32_t n_rows, int32_t n_cols, int32_t bdelta,
                                     const int32_t *mrow_ptr, const uint32_t *codes, const int8_t *q,
                                     const float *row_scale, const void *plan, const int32_t *tok_offsets,
                                     int32_t n_tok, float alpha, const uint16_t *x_f16, int64_t ldx, float beta, void *y,
                                     int32_t y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    return spmm_apply<true>(n_groups, n_rows, n_cols, bdelta, mrow_ptr, codes, q, row_scale, plan, tok_offsets, n_tok,
                            alpha, x_f16, ldx, beta, y, y_dtype, ldy, workspace, workspace_bytes, stream);
}
