// Weights of 4 bits with group scales on gfx950: the layout that the kernels
// read, the decoding into matrix-core operands, and a lane's piece of a row.
//
// Rows are taken 16 at a time (a matrix-core operand) and columns in blocks of
// 128.  The tile of 16 rows and a block is one record, in the order of the lanes
// that read it: 64 times 16 bytes of codes, lane l's those of row l % 16 and
// quarter l / 16, then 16 x groups scales and 16 x groups zero points.  (Row by
// row, as the weights come, the 16 lanes of a quarter touch 16 cache lines for 16
// bytes each: 8.3 M cache accesses for 12288 x 12288 and 28 us.)  A lane's 16
// bytes are its operands of the block's four 16x16x32 products: its word m holds
// columns 32 m + 8 (l / 16) .. + 7, so that product m covers the columns 32 m ..
// 32 m + 31 whole, and a group of 32, 64 or 128 columns is one, two or four
// products.  The weight's fragment is the second operand (D's columns are rows of
// W), the tokens' the first: a lane then decodes the row whose scale it multiplies
// with.
//
// Codes become exact 16-bit numbers (q - z) / UNIT (a code masked out of a word is
// the fp16 subnormal q 2^-24 or 16 q 2^-24, and one fused multiply-add brings it
// there).  The products of a group are summed in fp32 and multiplied with the
// group's scale in fp32: no weight is rounded.  The sums stay 1 / UNIT of the result
// until all are added and weighted, which costs one multiplication per result.  For
// fp16 UNIT is what that multiply-add leaves.  For bf16 it is 2^11: 128 products of
// the largest x with factors of 15, 1920 of them, stay finite where the scale brings
// the result back.  Such a sum is subnormal where the result is below 2^-115, and is
// rounded to multiples of 2^-138 of the result there; x, down to bf16's smallest
// number, is not.
#pragma once

#include "elem.hpp"

#include <type_traits>

namespace spmv {

typedef _Float16 q4_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 q4_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 q4_b2 __attribute__((ext_vector_type(2)));
typedef __bf16 q4_b8 __attribute__((ext_vector_type(8)));

constexpr int Q4_BLOCK = 128;      // columns of a block
constexpr int Q4_WORDS = 16;       // its words
constexpr int Q4_ROWS = 16;        // rows of a matrix-core operand

inline bool q4_group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }
inline int64_t q4_blocks(int64_t n_cols) { return ceil_div(n_cols, Q4_BLOCK); }
inline size_t q4_record(int32_t group, bool zeros) { return 1024 + (size_t)(Q4_BLOCK / group) * (zeros ? 48 : 32); }

// nibble of column e of a word's eight
__host__ __device__ constexpr int q4_place(int e) { return (e >> 1) + 4 * (e & 1); }

template <class E>
struct Q4Op;

template <>
struct Q4Op<F16> {
    typedef q4_h2 Zero;
    static constexpr float UNIT = 512.0f;      // what the sums are short of
    static __device__ __forceinline__ Zero zero(int z) {
        // z as the fp16 subnormal z 2^-24, times -2^15
        const q4_h2 s = __builtin_bit_cast(q4_h2, (unsigned)z * 0x00010001u);
        return s * q4_h2{(_Float16)-32768.0f, (_Float16)-32768.0f};
    }
    static __device__ __forceinline__ u32x4 decode(unsigned w, Zero nz) {
        const q4_h2 k0 = {(_Float16)32768.0f, (_Float16)32768.0f}, k1 = {(_Float16)2048.0f, (_Float16)2048.0f};
        const unsigned v = w >> 8;
        u32x4 o;
        o[0] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(q4_h2, w & 0x000F000Fu), k0, nz));
        o[1] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(q4_h2, w & 0x00F000F0u), k1, nz));
        o[2] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(q4_h2, v & 0x000F000Fu), k0, nz));
        o[3] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(q4_h2, v & 0x00F000F0u), k1, nz));
        return o;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(q4_h8, a), __builtin_bit_cast(q4_h8, b), c, 0, 0, 0);
    }
};

template <>
struct Q4Op<BF16> {
    typedef float Zero;
    static constexpr float UNIT = 2048.0f;
    static __device__ __forceinline__ Zero zero(int z) {
        // z as the fp16 subnormal z 2^-24, converted and multiplied by one instruction
        return __builtin_fmaf((float)__builtin_bit_cast(_Float16, (unsigned short)z), -16777216.0f / UNIT, 0.0f);
    }
    static __device__ __forceinline__ unsigned pair(unsigned bits, float k, Zero nz) {
        const q4_h2 h = __builtin_bit_cast(q4_h2, bits);
        q4_b2 r;
        r[0] = (__bf16)__builtin_fmaf((float)h[0], k, nz);
        r[1] = (__bf16)__builtin_fmaf((float)h[1], k, nz);
        return __builtin_bit_cast(unsigned, r);
    }
    static __device__ __forceinline__ u32x4 decode(unsigned w, Zero nz) {
        const unsigned v = w >> 8;
        u32x4 o;
        o[0] = pair(w & 0x000F000Fu, 8192.0f, nz);
        o[1] = pair(w & 0x00F000F0u, 512.0f, nz);
        o[2] = pair(v & 0x000F000Fu, 8192.0f, nz);
        o[3] = pair(v & 0x00F000F0u, 512.0f, nz);
        return o;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(q4_b8, a), __builtin_bit_cast(q4_b8, b), c, 0, 0, 0);
    }
};

// N bytes at any address.
template <int N>
struct Bytes {
    unsigned char b[N];
};
template <int N>
__device__ __forceinline__ Bytes<N> load_bytes(const void *p) {
    Bytes<N> r;
    __builtin_memcpy(&r, p, N);
    return r;
}

// Bytes of a record, and where its scales and zero points begin.
constexpr int Q4_SCALES = 1024;
template <bool ZP, int G>
struct Q4Rec {
    static constexpr int GB = Q4_BLOCK / G;        // groups of a block
    static constexpr int ZEROS = Q4_SCALES + 32 * GB;
    static constexpr int SIZE = ZEROS + (ZP ? 16 * GB : 0);
};

// A lane's place in the records of a row: of the 16 rows of a tile (the same base
// for all lanes, kept in scalar registers) or, tile by tile, of any row.
template <bool ZP, int G>
struct Q4Rows {
    const char *base;
    int lane, row;
    __device__ __forceinline__ Q4Rows() {}
    __device__ __forceinline__ Q4Rows(const char *tiles, int64_t tile, int n_blk)
        : base(tiles + tile * n_blk * Q4Rec<ZP, G>::SIZE), lane(__lane_id()), row(__lane_id() & 15) {}
    static __device__ __forceinline__ Q4Rows any(const char *tiles, int64_t r, int n_blk) {
        Q4Rows q(tiles, r >> 4, n_blk);
        q.row = (int)(r & 15);
        q.lane = (__lane_id() & 48) + q.row;
        return q;
    }
};

// A block of one row as a lane holds it: its quarter's codes, and the scales and zero
// points of all its groups.
template <class E, bool ZP, int G>
struct Q4Piece {
    static constexpr int GB = Q4_BLOCK / G;
    u32x4 c;
    Vec<E, GB> s;
    Bytes<ZP ? GB : 1> z;

    __device__ __forceinline__ void load(const Q4Rows<ZP, G> &rows, int b) {
        typedef Q4Rec<ZP, G> Rec;
        const char *rec = rows.base + (int64_t)b * Rec::SIZE;
        c = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(rec) + rows.lane);
        s = *(reinterpret_cast<const Vec<E, GB> *>(rec + Q4_SCALES) + rows.row);
        if constexpr (ZP) z = load_bytes<GB>(rec + Rec::ZEROS + rows.row * GB);
    }
    __device__ __forceinline__ float scale(int g) const { return (float)s.v[g]; }
    __device__ __forceinline__ int zero(int g) const {
        if constexpr (ZP)
            return z.b[g] & 15;
        else
            return 8;
    }
};

// 8 consecutive elements of a token's row from column c on, zeros past n_cols.
template <class T>
__device__ __forceinline__ u32x4 q4_token_piece(const T *row, int64_t c, int64_t n_cols) {
    if (c + 8 <= n_cols) return *reinterpret_cast<const u32x4_any *>(row + c);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < n_cols) {
            unsigned short h;
            __builtin_memcpy(&h, row + c + i, 2);
            v[i / 2] |= (unsigned)h << (16 * (i & 1));
        }
    return v;
}

// The same for the loops, in two steps (n_cols is at least 8): always one load, of
// the row's last 8 elements where column c is too far right, since a load under a
// condition makes every wait behind it wait for all loads; and, for the last block
// when it is used, what has been loaded moved to its place.
template <class T>
__device__ __forceinline__ u32x4 q4_token_ahead(const T *row, int c, int n_cols) {
    return *reinterpret_cast<const u32x4_any *>(row + min(c, n_cols - 8));
}
__device__ __forceinline__ u32x4 q4_token_placed(u32x4 v, int c, int n_cols) {
    typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
    const int drop = c - (n_cols - 8);                   // elements of columns before c
    if (drop <= 0) return v;
    u64x2 w = __builtin_bit_cast(u64x2, v);
    if (drop >= 4) w = u64x2{w[1], 0ull};
    const int s = 16 * (drop & 3);
    if (s) w = u64x2{w[0] >> s | w[1] << (64 - s), w[1] >> s};
    return drop >= 8 ? u32x4{0u, 0u, 0u, 0u} : __builtin_bit_cast(u32x4, w);
}

}  // namespace spmv
