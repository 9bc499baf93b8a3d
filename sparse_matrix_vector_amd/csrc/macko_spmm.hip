// MACKO products with many tokens on gfx950: y[t, :] = alpha * W x[t, :] + beta * y[t, :],
// for one pruned weight, or for one weight per group of sorted tokens.
//
// With one token the product is a gather (macko.hip).  With more, every
// decoded entry serves all tokens, so a piece of W is decoded into a dense
// fp16 tile in LDS, a slab of 256 columns at a time, and multiplied with the
// matrix cores (16x16x32, sums in fp32).  Two kernels: for few tokens a wave
// owns 16 rows and its tile, and waves never wait for each other
// (k_macko_spmm); for more, four waves share a tile of 64 rows and split the
// tokens (k_macko_spmm_block).  Sums are added in a fixed order everywhere.
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
// (One token with fp32 results goes to macko.hip's gather, which leaves pruned
// positions out.)
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
constexpr int SM_FRONT = 8;             // halfs before the first tile: spare columns of its first row
constexpr int SM_UNIT_BITS = 18;        // plan word: unit in the row, and how far back its predecessor's column lies
constexpr int SM_MAX_COLS = 1 << 20;    // (n_cols + 1024) / 8 units fit SM_UNIT_BITS

__device__ __forceinline__ f16x2 as_h2(unsigned int w) { return __builtin_bit_cast(f16x2, w); }

template <int BD>
struct Codes {
    typedef typename std::conditional<BD == 8, u32x2, unsigned int>::type lane_t;
    // the 8 codes of unit u (a word shared with 4 / BD - 1 neighbours for BD < 4)
    static __device__ __forceinline__ lane_t load(const unsigned int *__restrict__ codes, unsigned int u) {
        const char *p = reinterpret_cast<const char *>(codes) + (BD < 4 ? (u * BD) & ~3u : u * BD);
        return *reinterpret_cast<const lane_t *>(p);
    }
    // inclusive prefix of (code + 1) over the unit's entries
    static __device__ __forceinline__ void prefix(lane_t w, unsigned int u, int (&p)[8]) {
        int run = 0;
        if constexpr (BD == 8) {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                run += (int)(((t < 4 ? w.x : w.y) >> (8 * (t & 3))) & 255u) + 1;
                p[t] = run;
            }
        } else {
            const unsigned int ws = BD < 4 ? w >> ((8 * BD * u) & 31u) : w;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                run += (int)((ws >> (BD * t)) & ((1u << BD) - 1u)) + 1;
                p[t] = run;
            }
        }
    }
};

// the unit's 8 values: 16 bytes of fp16 or 8 bytes of int8 (fewer than 2^31
// entries: byte offsets fit 32 bits)
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

// The streamed arrays as buffers: a lane whose offset lies past the end reads
// zeros without a memory access, so lanes without a unit cost nothing and need
// no branch.  (Sizes are below 4 GB: fewer than 2^31 entries, in units of 128.)
struct Streams {
    __amdgpu_buffer_rsrc_t codes, vals;
};
constexpr unsigned int SM_NO_UNIT = 0xFFFFFFF0u;

template <int BD, bool I8>
__device__ __forceinline__ Streams streams_of(const unsigned int *codes, const void *vals, int units) {
    constexpr int FLAGS = 0x00027000;
    return {__builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned int *>(codes), 0, (int)((unsigned)units * BD), FLAGS),
            __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(vals), 0,
                                              (int)((unsigned)units * (unsigned)sizeof(vals_t<I8>)), FLAGS)};
}
template <int BD>
__device__ __forceinline__ typename Codes<BD>::lane_t stream_codes(const Streams &s, bool in, unsigned int u) {
    const int at = (int)(in ? (BD < 4 ? (u * BD) & ~3u : u * BD) : SM_NO_UNIT);
    if constexpr (BD == 8)
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(s.codes, at, 0, 0));
    else
        return __builtin_amdgcn_raw_buffer_load_b32(s.codes, at, 0, 0);
}
template <bool I8>
__device__ __forceinline__ vals_t<I8> stream_vals(const Streams &s, bool in, unsigned int u) {
    const int at = (int)(in ? u * (unsigned)sizeof(vals_t<I8>) : SM_NO_UNIT);
    if constexpr (I8)
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(s.vals, at, 0, 0));
    else
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(s.vals, at, 0, 0));
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

// Plan: one wave per row walks the row's units 64 at a time.  Built once per
// weight; it reads the codes: 15 to 25 us for 12288 x 12288, half kept.
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
        Codes<BD>::prefix(in ? Codes<BD>::load(codes, (unsigned)(u0 + b + lane)) : typename Codes<BD>::lane_t{},
                          (unsigned)(u0 + b + lane), p);
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

// y[tok, r .. r + 3] from the sums v of those rows (global rows `row` ..).
template <bool I8>
__device__ __forceinline__ void finish(const SpmmArg &a, int tok, int r, int64_t row, f32x4 v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= I8 && r + j < a.n_rows ? a.alpha * a.row_scale[row + j] : a.alpha;
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

// A wave's 16 rows, 8 at a time (h = 0, 1); lane l of a row's 8 lanes takes
// every eighth unit of the row's piece of a slab.
struct RowPair {
    int base[2], units[2];      // first unit and number of units of the rows
    const unsigned int *plan[2];
};

// Rows past the end of the group count as empty.
__device__ __forceinline__ RowPair load_rows(const SpmmArg &a, int64_t row0, int rows, int lane) {
    RowPair rp;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + (lane >> 3);
        const int64_t row = row0 + max(min(r, rows - 1), 0);
        const int b = a.mrp[row] / 8, e = a.mrp[row + 1] / 8;
        rp.units[h] = r < rows ? e - b : 0;
        rp.base[h] = b;
        rp.plan[h] = a.plan + row * (a.n_slabs + 1);
    }
    return rp;
}

// The units of one slab in registers: SM_STEPS of 8 lanes cover a slab of a
// half pruned row, further ones are loaded while decoding.  No load hides
// behind a branch, so they stay in flight over other work.  (Two steps: 12288 x
// 12288 times 2 to 128, 30 % kept, 2 to 7 % faster; half kept times 513, 445
// against 422 us.)
constexpr int SM_STEPS = 3;
template <int BD, bool I8>
struct Stage {
    int u[2], end[2], carry[2];
    typename Codes<BD>::lane_t w[2][SM_STEPS];
    vals_t<I8> v[2][SM_STEPS];
};

struct PlanWords {
    unsigned int p0[2], p1[2];
};

__device__ __forceinline__ PlanWords load_plan(const RowPair &rp, int k) {
    PlanWords w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w.p0[h] = rp.plan[h][k];
        w.p1[h] = rp.plan[h][k + 1];
    }
    return w;
}

template <int BD, bool I8>
__device__ __forceinline__ void load_half(Stage<BD, I8> &st, const Streams &a, const RowPair &rp, const PlanWords &w, int l,
                                          int h) {
    {
        st.u[h] = (int)(w.p0[h] & ((1u << SM_UNIT_BITS) - 1u)) + l;
        st.end[h] = min((int)(w.p1[h] & ((1u << SM_UNIT_BITS) - 1u)) + 1, rp.units[h]);
        st.carry[h] = -1 - (int)(w.p0[h] >> SM_UNIT_BITS);      // relative to the slab's first column
#pragma unroll
        for (int i = 0; i < SM_STEPS; ++i) {
            const bool in = st.u[h] + 8 * i < st.end[h];
            const unsigned int u = (unsigned)(rp.base[h] + st.u[h] + 8 * i);
            st.w[h][i] = stream_codes<BD>(a, in, u);
            st.v[h][i] = stream_vals<I8>(a, in, u);
        }
    }
}

template <int BD, bool I8>
__device__ __forceinline__ void load_stage(Stage<BD, I8> &st, const Streams &a, const RowPair &rp, const PlanWords &w,
                                           int l) {
    load_half<BD, I8>(st, a, rp, w, l, 0);
    load_half<BD, I8>(st, a, rp, w, l, 1);
}

// Byte offsets 2 * (code sums + entries so far) of the unit's 8 entries, and
// the unit's whole advance in columns.  4-bit codes are summed as bytes: even
// and odd codes apart, doubled, then two shifted adds give all prefix sums
// (at most 240, so no carries; the last entry's offset, up to 256, is the total).
template <int BD>
__device__ __forceinline__ int unit_offsets(typename Codes<BD>::lane_t w, unsigned int unit, int (&o)[8]) {
    if constexpr (BD == 4) {
        const unsigned int lo = (w << 1) & 0x1E1E1E1Eu, hi = (w >> 3) & 0x1E1E1E1Eu;
        unsigned int P = lo + hi;
        asm volatile("" : "+v"(P));           // shifted adds stay adds (not quarter-rate multiplies)
        P += P << 8;
        asm volatile("" : "+v"(P));
        P += P << 16;
        asm volatile("" : "+v"(P));
        const unsigned int E = (P << 8) + lo + 0x0E0A0602u;   // entries 0, 2, 4, 6
        const unsigned int Q = P + 0x000C0804u;               // entries 1, 3, 5
        const int tot = (int)(P >> 25) + 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[2 * k] = (int)((E >> (8 * k)) & 255u);
            o[2 * k + 1] = k < 3 ? (int)((Q >> (8 * k)) & 255u) : 2 * tot;
        }
        return tot;
    } else {
        Codes<BD>::prefix(w, unit, o);
        const int tot = o[7];
#pragma unroll
        for (int t = 0; t < 8; ++t) o[t] *= 2;
        return tot;
    }
}

typedef __attribute__((address_space(3))) unsigned short lds_half;
__device__ __forceinline__ int lds_offset(const unsigned short *p) {
    return (int)(uintptr_t)(const __attribute__((address_space(3))) unsigned short *)p;
}
__device__ __forceinline__ int clamp3(int v, int lo, int hi) {
    int r;
    asm("v_med3_i32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "v"(lo), "v"(hi));
    return r;
}

// One step: the 8 lanes of each row decode 8 units into the tile row at `row`
// (LDS byte offset).  Entries of neighbouring slabs are clamped into the spare
// columns on both sides of the row.
template <int BD, bool I8>
__device__ __forceinline__ void decode_step(typename Codes<BD>::lane_t w, const vals_t<I8> &v, unsigned int unit, bool in,
                                            int &carry, int odd, int high, int row) {
    int o[8];
    const int all = unit_offsets<BD>(w, unit, o);
    const int tot = in ? all : 0;
    int incl = scan8(tot, odd, high);
    asm volatile("" : "+v"(incl));
    const int before = row + 2 * (carry + incl - tot);
    carry += last8(incl);
    if (in) {
        const int lo = row - 2, hi = row + 2 * SM_SLAB;
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            const unsigned int h = value_pair<I8>(v, t);
            *(lds_half *)(uintptr_t)(unsigned)clamp3(before + o[t], lo, hi) = (unsigned short)h;
            *(lds_half *)(uintptr_t)(unsigned)clamp3(before + o[t + 1], lo, hi) = (unsigned short)(h >> 16);
        }
    }
}

// Eight of the wave's rows of a slab into its tile at `tile` (LDS byte offset).
template <int BD, bool I8>
__device__ __forceinline__ void decode_half(Stage<BD, I8> &st, const Streams &a, const RowPair &rp, int lane, int tile,
                                            int h) {
    const int odd = lane & 1 ? -1 : 0, high = lane & 2 ? -1 : 0;
    {
        const int row = tile + 2 * (8 * h + (lane >> 3)) * SM_LDW;
#pragma unroll
        for (int i = 0; i < SM_STEPS; ++i) {
            const int u = st.u[h] + 8 * i;
            if (i > 0 && !__any(u < st.end[h])) break;
            decode_step<BD, I8>(st.w[h][i], st.v[h][i], (unsigned)(rp.base[h] + u), u < st.end[h], st.carry[h], odd, high,
                                row);
        }
        for (int u = st.u[h] + 8 * SM_STEPS; __any(u < st.end[h]); u += 8) {
            const unsigned int at = (unsigned)(rp.base[h] + u);
            const bool in = u < st.end[h];
            decode_step<BD, I8>(stream_codes<BD>(a, in, at), stream_vals<I8>(a, in, at), at, in, st.carry[h], odd, high, row);
        }
    }
}

template <int BD, bool I8>
__device__ __forceinline__ void decode_stage(Stage<BD, I8> &st, const Streams &a, const RowPair &rp, int lane, int tile) {
    decode_half<BD, I8>(st, a, rp, lane, tile, 0);
    decode_half<BD, I8>(st, a, rp, lane, tile, 1);
}

// Clears the 256 columns of a wave's 16 rows: each half wave a row per store.
__device__ __forceinline__ void clear_tile(unsigned short *tile, int lane) {
    unsigned short *p = tile + (lane >> 5) * SM_LDW + 8 * (lane & 31);
#pragma unroll
    for (int i = 0; i < SM_ROWS; i += 2) *reinterpret_cast<u32x4 *>(p + i * SM_LDW) = u32x4{0u, 0u, 0u, 0u};
}

// Few tokens, 32 at most.  Workgroup: rows 16 blockIdx.x .. of group blockIdx.y and
// that group's tokens, slabs wave, wave + WAVES, ...; the waves add their sums at
// the end.  Bound by the latency of a slab's chain (plan word,
// codes, scan, LDS, product), so small calls want many waves.  5.7 us for
// 2048 x 2048 (half kept) times 5, of which about 3 are the launch; 38 us
// for 12288 x 12288 (30 % kept) times 2, 116 MB at 3.0 TB/s.
template <int BD, bool I8, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_macko_spmm(SpmmArg a) {
    static_assert(NT <= 2, "x is held in registers for a whole slab");
    extern __shared__ __attribute__((aligned(16))) unsigned short lds[];
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int t0 = 0, t1 = a.n_tok;
    if (a.tok_offsets) {
        t0 = min(max(a.tok_offsets[blockIdx.y], 0), a.n_tok);
        t1 = min(max(a.tok_offsets[blockIdx.y + 1], t0), a.n_tok);
    }
    if (t0 >= t1) return;
    const int live = min(NT, (t1 - t0 + 15) / 16);      // token tiles in use
    const int r0 = blockIdx.x * SM_ROWS;
    const int rows = min(SM_ROWS, a.n_rows - r0);
    const int64_t row0 = (int64_t)blockIdx.y * a.n_rows + r0;
    unsigned short *tile = lds + SM_FRONT + wv * SM_ROWS * SM_LDW;
    const unsigned short *xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = a.x + (int64_t)min(t0 + 16 * i + n, t1 - 1) * a.ldx;
    f32x4 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const Streams str = streams_of<BD, I8>(a.codes, a.vals, a.mrp[(int64_t)gridDim.y * a.n_rows] / 8);
    const RowPair rp = load_rows(a, row0, rows, lane);
    // one slab: its units are in st; next gets those of slab k + WAVES, whose
    // plan words are in pw, and pw those of the slab after that
    PlanWords pw;
    const int top = wv + (a.n_slabs - 1 - wv) / WAVES * WAVES;   // the wave's last slab, read again at the end
    auto slab = [&](int k, Stage<BD, I8> &st, Stage<BD, I8> &next) {
        // loads are waited for in the order of their issue: what is needed
        // first goes first, and the next slab's units last
        // columns past the last are read as the row's last ones: W is zero there
        const int c0 = k * SM_SLAB + 8 * q, cm = a.n_cols - 8;
        u32x4 x[NT][8];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int s = 0; s < 8; ++s)
                x[i][s] = *reinterpret_cast<const u32x4 *>(xr[i] + min(c0 + 32 * s, cm));
        const PlanWords after = load_plan(rp, min(k + 2 * WAVES, top));
        __builtin_amdgcn_sched_barrier(0);
        load_stage<BD, I8>(next, str, rp, pw, lane & 7);
        __builtin_amdgcn_sched_barrier(0);
        pw = after;
        clear_tile(tile, lane);
        wave_lds_order();
        decode_stage<BD, I8>(st, str, rp, lane, lds_offset(tile));
        wave_lds_order();
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const h8 w = __builtin_bit_cast(
                h8, *reinterpret_cast<const u32x4 *>(tile + n * SM_LDW + 32 * s + 8 * q));
#pragma unroll
            for (int i = 0; i < NT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(h8, x[i][s]), acc[i], 0, 0, 0);
        }
        wave_lds_order();
    };
    if (wv < a.n_slabs) {
        Stage<BD, I8> s0, s1;
        const PlanWords first = load_plan(rp, wv);
        pw = load_plan(rp, min(wv + WAVES, top));
        __builtin_amdgcn_sched_barrier(0);
        load_stage<BD, I8>(s0, str, rp, first, lane & 7);
        int k = wv;
        for (; k + WAVES < a.n_slabs; k += 2 * WAVES) {
            slab(k, s0, s1);
            slab(k + WAVES, s1, s0);
        }
        if (k < a.n_slabs) slab(k, s0, s1);
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
        const int tok = t0 + 16 * i + n;                 // D: row 4 q + j, column (token) n
        if (tok < t1) finish<I8>(a, tok, r0 + 4 * q, row0 + 4 * q, v);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: 64 rows of W per workgroup, each of 4 waves decoding 16 of them
// into a common tile and multiplying all 64 by tokens of its own, so x goes
// from memory straight to the registers of the one wave that uses it, and a W
// operand read from LDS serves all of the wave's tokens.  With fewer than four
// token tiles the waves of one tile share out its columns instead.
//
// Per slab a workgroup clears 33 KB of LDS, scatters its entries two bytes at a
// time and reads the tile once per wave; with decoding's integer work these
// take turns between two barriers, hidden only by the CU's other workgroups.
// 12288 x 12288, 30 % kept: 46 us times 32 (116 MB at 2.5 TB/s).  Half kept,
// int8: 420 us times 513 (369 TFLOP/s counting every position): x comes from
// L2 once per 64 rows, 2.4 GB.  Measured and not kept: x through LDS (580),
// 128 rows per workgroup (495), two W tiles in turn (432 + join).
// ---------------------------------------------------------------------------
template <int NT>
struct BlockShape {
    static constexpr int WAVES = 4;
    static constexpr int ROWS = WAVES * SM_ROWS;
    static constexpr int TILE = ROWS * SM_LDW;              // halfs
    static constexpr int KW = NT < 4 ? 4 / NT : 1;          // waves that share out a token tile's columns
    static constexpr int GROUPS = 4 / KW;                   // of KW waves, each with every GROUPS-th token tile
    static constexpr int TW = NT / GROUPS;                  // token tiles of a wave
    static constexpr int STEPS = 8 / KW;                    // 32-column steps of a wave per slab
    static constexpr int AHEAD = STEPS * TW <= 16 ? STEPS : 16 / TW;   // steps of x in registers
    static constexpr int OCC = NT < 8 ? 4 : 2;              // waves per SIMD that the registers allow
    // the tile, or the column parts' sums
    static constexpr size_t LDS = std::max<size_t>((size_t)(SM_FRONT + TILE) * 2, (size_t)(KW - 1) * NT * 4 * 64 * 16);
};

// an LDS-only barrier: loads issued before it stay in flight
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A workgroup takes 64 rows of a group, one of `split` parts of its slabs, and
// `width` 16-token tiles; row blocks first, so that workgroups that run together
// share the piece of x.  (Runs of row blocks per XCD measured 2 % slower.)
template <int BD, bool I8, int NT>
__global__ __launch_bounds__(64 * BlockShape<NT>::WAVES, BlockShape<NT>::OCC) void k_macko_spmm_block(SpmmArg a, int n_groups, int row_blocks, int tiles, int width, int split,
                                                                       float *__restrict__ partial, int ldp) {
    typedef BlockShape<NT> B;
    extern __shared__ __attribute__((aligned(16))) unsigned short lds[];
    const int lane = __lane_id(), q = lane >> 4, n = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int rb = (int)(blockIdx.x % (unsigned)row_blocks);
    int rest = (int)(blockIdx.x / (unsigned)row_blocks);
    const int tt = rest % tiles;
    rest /= tiles;
    const int part = rest % split, group = rest / split;
    int t0 = 0, t1 = a.n_tok;
    if (a.tok_offsets) {
        t0 = min(max(a.tok_offsets[group], 0), a.n_tok);
        t1 = min(max(a.tok_offsets[group + 1], t0), a.n_tok);
    }
    t0 += tt * 16 * width;
    if (t0 >= t1) return;
    t1 = min(t1, t0 + 16 * width);
    const int r0 = rb * B::ROWS;
    const int64_t row0 = (int64_t)group * a.n_rows + r0;
    const int kp = wv / B::GROUPS, tw0 = wv % B::GROUPS;    // the wave's part of the columns, first token tile
    const int live = (t1 - t0 + 15) / 16;                   // token tiles in use
    const int mine = min(B::TW, max(0, (live - tw0 + B::GROUPS - 1) / B::GROUPS));
    const int wrow = wv * SM_ROWS;                          // the wave's rows in the decoding
    unsigned short *tile = lds + SM_FRONT + wrow * SM_LDW;
    f32x4 acc[4][B::TW];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < B::TW; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const Streams str = streams_of<BD, I8>(a.codes, a.vals, a.mrp[(int64_t)n_groups * a.n_rows] / 8);
    const RowPair rp = load_rows(a, row0 + min(wrow, a.n_rows - 1 - r0), a.n_rows - r0 - wrow, lane);
    const unsigned short *xr[B::TW];
#pragma unroll
    for (int t = 0; t < B::TW; ++t)
        xr[t] = a.x + (int64_t)min(t0 + 16 * (tw0 + B::GROUPS * t) + n, t1 - 1) * a.ldx;
    // at least one slab: split is at most their number
    const int lo = (int)((int64_t)a.n_slabs * part / split), hi = (int)((int64_t)a.n_slabs * (part + 1) / split);
    const int cm = a.n_cols - 8;
    const int col = kp * 32 * B::STEPS + 8 * q;         // the lane's first column in a slab
    u32x4 x[B::AHEAD][B::TW];
    // columns past the last are read as the row's last ones: W is zero there
    auto load_x = [&](int k, int s, int slot) {
#pragma unroll
        for (int t = 0; t < B::TW; ++t)
            x[slot][t] = *reinterpret_cast<const u32x4 *>(xr[t] + min(k * SM_SLAB + col + 32 * s, cm));
    };
    Stage<BD, I8> st;
    const PlanWords first = load_plan(rp, lo);
    PlanWords pw = load_plan(rp, min(lo + 1, hi - 1));
    __builtin_amdgcn_sched_barrier(0);
    load_stage<BD, I8>(st, str, rp, first, lane & 7);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < B::AHEAD; ++s) load_x(lo, s, s);
    for (int k = lo; k < hi; ++k) {
        clear_tile(tile, lane);
        wave_lds_order();
        // half by half, the next slab's units are loaded as soon as their
        // registers are free; the next x is in flight over the decoding
        const PlanWords after = load_plan(rp, min(k + 2, hi - 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            decode_half<BD, I8>(st, str, rp, lane, lds_offset(tile), h);
            __builtin_amdgcn_sched_barrier(0);
            load_half<BD, I8>(st, str, rp, pw, lane & 7, h);
            __builtin_amdgcn_sched_barrier(0);
        }
        pw = after;
        lds_barrier();
#pragma unroll
        for (int s = 0; s < B::STEPS; ++s) {
            h8 w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[r] = __builtin_bit_cast(h8, *reinterpret_cast<const u32x4 *>(lds + SM_FRONT + (16 * r + n) * SM_LDW +
                                                                               (kp * B::STEPS + s) * 32 + 8 * q));
#pragma unroll
            for (int t = 0; t < B::TW; ++t) {
                if (t < mine) {                         // uniform
                    const h8 xv = __builtin_bit_cast(h8, x[s % B::AHEAD][t]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[r], xv, acc[r][t], 0, 0, 0);
                }
            }
            if (s + B::AHEAD < B::STEPS)
                load_x(k, s + B::AHEAD, s % B::AHEAD);
            else
                load_x(min(k + 1, hi - 1), (s + B::AHEAD) % B::STEPS, s % B::AHEAD);
        }
        lds_barrier();
    }
    if (B::KW > 1) {                                        // the column parts, in order
        f32x4 *sums = reinterpret_cast<f32x4 *>(lds) + tw0 * (4 * B::TW * 64) + lane;   // [KW - 1][GROUPS][TW][4][64]
        constexpr int PART = B::GROUPS * B::TW * 4 * 64;
        __syncthreads();
        if (kp > 0) {
#pragma unroll
            for (int t = 0; t < B::TW; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) sums[(kp - 1) * PART + (t * 4 + r) * 64] = acc[r][t];
        }
        __syncthreads();
        if (kp > 0) return;
#pragma unroll
        for (int p = 0; p < B::KW - 1; ++p)
#pragma unroll
            for (int t = 0; t < B::TW; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r][t] += sums[p * PART + (t * 4 + r) * 64];
    }
#pragma unroll
    for (int t = 0; t < B::TW; ++t) {
        const int tok = t0 + 16 * (tw0 + B::GROUPS * t) + n;
        if (tok >= t1) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = r0 + 16 * r + 4 * q;
            if (row >= a.n_rows) continue;
            if (split > 1)
                *reinterpret_cast<f32x4 *>(partial + ((int64_t)part * a.n_tok + tok) * ldp + row) = acc[r][t];
            else
                finish<I8>(a, tok, row, row0 - r0 + row, acc[r][t]);
        }
    }
}

// Adds the parts of k_macko_spmm_block in order; bound by their traffic (513
// tokens of 12288 rows: 20 us).
template <bool I8>
__global__ __launch_bounds__(256) void k_macko_spmm_join(SpmmArg a, int n_groups, int split,
                                                         const float *__restrict__ partial, int ldp) {
    const int r = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (r >= a.n_rows) return;
    int t0 = 0, t1 = a.n_tok;
    if (a.tok_offsets) {
        t0 = min(max(a.tok_offsets[0], 0), a.n_tok);
        t1 = min(max(a.tok_offsets[n_groups], t0), a.n_tok);
    }
    for (int tok = t0 + blockIdx.y; tok < t1; tok += gridDim.y) {
        f32x4 v = *reinterpret_cast<const f32x4 *>(partial + (int64_t)tok * ldp + r);
        for (int s = 1; s < split; ++s)
            v += *reinterpret_cast<const f32x4 *>(partial + ((int64_t)s * a.n_tok + tok) * ldp + r);
        int64_t row = r;
        if (I8 && n_groups > 1) {                           // the token's group
            int g = 0;
            while (g + 1 < n_groups && a.tok_offsets[g + 1] <= tok) ++g;
            row += (int64_t)g * a.n_rows;
        }
        finish<I8>(a, tok, r, row, v);
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
    const size_t lds = std::max<size_t>((size_t)(SM_FRONT + WAVES * SM_ROWS * SM_LDW) * 2, (size_t)WAVES * NT * 64 * 16);
    k_macko_spmm<BD, I8, NT, WAVES><<<grid, 64 * WAVES, lds, st>>>(a);
}

// How the tokens and columns of a product are cut.
struct Cut {
    bool block;       // k_macko_spmm_block, else k_macko_spmm
    int waves;        // of a workgroup of k_macko_spmm
    int nt;           // token tiles a workgroup can hold
    int width;        // token tiles it takes
    int tiles;        // workgroups over the tokens (of the largest possible group)
    int split;        // workgroups over the columns
};

Cut cut_of(int64_t n_groups, int64_t n_rows, int64_t n_cols, int64_t n_tok, int64_t max_split = 16) {
    Cut c = {};
    const int64_t t16 = std::max<int64_t>(1, ceil_div(n_tok, 16));
    // Up to 32 tokens, as long as the traffic of x (every 16 rows read all of it)
    // is small: 12288 x 12288 at 70 % measured 41.5 against 45.9 us in 64-row
    // workgroups for 8 tokens (151 MB of x), 53.0 against 48.4 us for 16 (302 MB).
    // Above 16 tokens only up to 24 slabs: 4096 x 4096 times 32 takes 14.5 against
    // 19.6 us, but 1024 x 12288 takes 31 against 15.5 us with its columns split.
    const int64_t slabs = ceil_div(n_cols, SM_SLAB);
    c.block = n_tok > 32 || (n_tok > 16 && slabs > 24) || ceil_div(n_rows, SM_ROWS) * n_tok * n_cols * 2 > (200 << 20);
    if (!c.block) {
        // few row tiles: more waves share a tile's slabs (2048 x 2048 times 5:
        // 5.3 us with 8, 6.7 us with 4; 8192 x 8192 times 2: 23.1 and 20.9 us)
        c.waves = n_groups * ceil_div(n_rows, SM_ROWS) <= 256 && slabs >= 8 ? 8 : 4;
        c.nt = (int)t16;
        c.tiles = c.split = 1;
        c.width = c.nt;
        return c;
    }
    // a group's share of the tokens is not known here: room for twice the mean
    // (8 groups of 4096 x 2048, 30 % kept, in random shares: 400 tokens 33 us, 47 with
    // room for the mean; 1000 tokens 54 and 77; 600 tokens 43 and 38)
    const int64_t room = n_groups > 1 ? std::min(t16, ceil_div(2 * n_tok, 16 * n_groups)) : t16;
    c.nt = room > 8 ? 16 : room > 4 ? 8 : room > 2 ? 4 : 2;
    c.tiles = (int)ceil_div(t16, c.nt);
    c.width = n_groups > 1 ? c.nt : (int)ceil_div(t16, c.tiles);
    c.split = 1;
    // Parts of the columns, by an estimate of the time in us: a slab takes
    // longer the more workgroups share a CU (`alone` + `each` per resident one,
    // rough figures of this kernel's own times), starting a workgroup is counted
    // as two slabs, joining as a launch and the traffic of the parts' sums at
    // 4 TB/s.  Against counting rounds of slabs only: 4096 x 4096, 10 % kept, 64
    // tokens 26.3 -> 16.3 us (16 parts were too many); 12288 x 12288, 30 % kept,
    // 64 tokens 68.7 -> 63.0, 128 tokens 116.8 -> 105.6; 513 tokens the same.
    const int fit = c.nt < 8 ? 4 : 2;                       // workgroups per CU
    const double alone = c.nt == 2 ? 0.8 : c.nt == 4 ? 1.0 : c.nt == 8 ? 1.2 : 1.9;
    const double each = c.nt == 2 ? 0.95 : c.nt == 4 ? 1.0 : c.nt == 8 ? 1.5 : 2.2;
    double best = 1e30;
    for (int s = 1; s <= 16 && s <= slabs && (s == 1 || s <= max_split); ++s) {
        const int64_t wgs = n_groups * ceil_div(n_rows, BlockShape<4>::ROWS) * c.tiles * s, full = wgs / (256 * fit);
        const int64_t rest = ceil_div(wgs - full * 256 * fit, 256);
        const double slab = (double)full * (alone + each * fit) + (rest ? alone + each * (double)rest : 0.0);
        const double cost = slab * (double)(ceil_div(slabs, s) + 2) +
                            (s > 1 ? 4.0 + s * (double)n_tok * (double)n_rows * 2e-6 : 0.0);
        if (cost < best) best = cost, c.split = s;
    }
    return c;
}

int64_t partial_ld(int64_t n_rows) { return ceil_div(n_rows, 4) * 4; }

size_t packed_bytes(int64_t n_tok, int64_t n_cols) {
    return ((size_t)n_tok * (size_t)(ceil_div(n_cols, 8) * 8) * 2 + 15) & ~size_t(15);
}

// the sums of one part of the columns
size_t part_bytes(int64_t n_tok, int64_t n_rows) { return (size_t)n_tok * (size_t)partial_ld(n_rows) * 4; }

template <int BD, bool I8, int NT>
spmv_status launch_block(const SpmmArg &a, const Cut &c, int n_groups, float *partial, hipStream_t st) {
    const int row_blocks = (int)ceil_div(a.n_rows, BlockShape<NT>::ROWS);
    const int64_t grid = (int64_t)row_blocks * c.tiles * c.split * n_groups;
    const spmv_status fits = check_grid(grid, 64 * BlockShape<NT>::WAVES);
    if (fits != SPMV_OK) return fits;
    k_macko_spmm_block<BD, I8, NT><<<(unsigned)grid, 64 * BlockShape<NT>::WAVES, BlockShape<NT>::LDS, st>>>(
        a, n_groups, row_blocks, c.tiles, c.width, c.split, partial, (int)partial_ld(a.n_rows));
    SPMV_LAUNCHED("k_macko_spmm_block");
    return SPMV_OK;
}

template <int BD, bool I8, int NT>
void launch_waves(const SpmmArg &a, const Cut &c, dim3 grid, hipStream_t st) {
    if (c.waves == 8)
        launch<BD, I8, NT, 8>(a, grid, st);
    else
        launch<BD, I8, NT, 4>(a, grid, st);
}

template <int BD, bool I8>
spmv_status launch_shape(const SpmmArg &a, const Cut &c, int n_groups, float *partial, hipStream_t st) {
    if (!c.block) {
        const dim3 grid((unsigned)ceil_div(a.n_rows, SM_ROWS), n_groups);
        if (c.nt == 1)
            launch_waves<BD, I8, 1>(a, c, grid, st);
        else
            launch_waves<BD, I8, 2>(a, c, grid, st);
        SPMV_LAUNCHED("k_macko_spmm");
        return SPMV_OK;
    }
    spmv_status s;
    switch (c.nt) {
        case 2: s = launch_block<BD, I8, 2>(a, c, n_groups, partial, st); break;
        case 4: s = launch_block<BD, I8, 4>(a, c, n_groups, partial, st); break;
        case 8: s = launch_block<BD, I8, 8>(a, c, n_groups, partial, st); break;
        default: s = launch_block<BD, I8, 16>(a, c, n_groups, partial, st); break;
    }
    if (s != SPMV_OK) return s;
    if (c.split > 1) {
        k_macko_spmm_join<I8><<<dim3((unsigned)ceil_div(a.n_rows, 1024), (unsigned)std::min(a.n_tok, 65535)), 256, 0, st>>>(
            a, n_groups, c.split, partial, (int)partial_ld(a.n_rows));
        SPMV_LAUNCHED("k_macko_spmm_join");
    }
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
    if (n_groups > 4095 || ceil_div(n_rows, SM_ROWS) > 65535)
        return fail(SPMV_ERR_UNSUPPORTED, "more than 4095 groups or %d rows are not supported", 65535 * SM_ROWS);
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
    // one token is the vector product, whose gather of x needs no dense tile
    // (12288 x 12288 at 70 %: 20.5 us against 34); it writes fp32 only
    if (n_tok == 1 && !tok_offsets && y_dtype == SPMV_F32) {
        if constexpr (I8)
            return macko_spmv_i8(n_rows, n_cols, bdelta, mrow_ptr, codes, static_cast<const int8_t *>(vals), row_scale, alpha,
                                 x, beta, static_cast<float *>(y), stream);
        else
            return macko_spmv(n_rows, n_cols, bdelta, mrow_ptr, codes, static_cast<const uint16_t *>(vals), alpha, x, beta,
                              static_cast<float *>(y), stream);
    }
    // the workspace: x packed where that is needed, then as many parts as fit
    // (the best cut of a smaller batch may want more than a larger one's)
    const bool pack = !aligned16(x) || ldx % 8 != 0 || n_cols % 8 != 0;
    const size_t packed = pack ? packed_bytes(n_tok, n_cols) : 0;
    if (pack && (!workspace || workspace_bytes < packed))
        return fail(SPMV_ERR_INVALID_VALUE, "x of this shape and alignment needs a workspace of %zu bytes", packed);
    const size_t room = workspace && workspace_bytes > packed ? workspace_bytes - packed : 0;
    const Cut cut = cut_of(n_groups, n_rows, n_cols, n_tok, (int64_t)std::min<size_t>(16, room / part_bytes(n_tok, n_rows)));
    if ((pack || cut.split > 1) && !aligned16(workspace))
        return fail(SPMV_ERR_INVALID_VALUE, "workspace must be 16-byte aligned");
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + packed);
    if (pack) {
        const int ldp = (int)(ceil_div(n_cols, 8) * 8);
        k_macko_spmm_pack<<<dim3((unsigned)ceil_div(ldp, 256), (unsigned)std::min(n_tok, 65535)), 256, 0, s>>>(
            n_tok, n_cols, ldp, x, ldx, static_cast<unsigned short *>(workspace));
        SPMV_LAUNCHED("k_macko_spmm_pack");
        a.x = static_cast<const unsigned short *>(workspace);
        a.ldx = ldp;
        a.n_cols = ldp;
    }
    switch (bdelta) {
        case 1: return launch_shape<1, I8>(a, cut, n_groups, partial, s);
        case 2: return launch_shape<2, I8>(a, cut, n_groups, partial, s);
        case 4: return launch_shape<4, I8>(a, cut, n_groups, partial, s);
        default: return launch_shape<8, I8>(a, cut, n_groups, partial, s);
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

extern "C" spmv_status macko_spmm_workspace_size(int32_t n_groups, int32_t n_rows, int32_t n_cols, int32_t n_tok,
                                                 size_t *bytes) {
    if (!bytes) return fail(SPMV_ERR_INVALID_VALUE, "bytes is NULL");
    if (n_groups < 1 || n_tok < 0) return fail(SPMV_ERR_INVALID_VALUE, "n_groups must be >= 1 and n_tok >= 0");
    const spmv_status st = check_size(n_rows, n_cols);
    if (st != SPMV_OK) return st;
    const Cut c = cut_of(n_groups, n_rows, n_cols, n_tok);
    *bytes = packed_bytes(n_tok, n_cols) +
             (c.split > 1 ? (size_t)c.split * part_bytes(n_tok, n_rows) : 0);
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
