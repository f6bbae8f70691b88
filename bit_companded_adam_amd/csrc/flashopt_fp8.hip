// Matrices in 8 bits: E4M3 or E5M2 codes with one E8M0 scale for each 128
// elements along a row, or for each block of 128 x 128 (flashopt_byte_quantize,
// flashopt_byte_dequantize), and the product of two such matrices
// (flashopt_byte_product, flashopt_byte_linear).
//
// Storage of an R x C matrix: codes, R rows of Cp = 128 ceil(C / 128) bytes, so
// that a group is one 128-byte line and one K step of a matrix instruction;
// scales, R rows of ceil(C / 128) bytes padded to a multiple of 16, so that
// sixteen steps' scales are one aligned load.  Padding is zero.  A scale of a
// block of 128 x 128 stands in each of its rows: the product knows one kind of
// operand, and a weight and its transpose stand for the same values.
//
// Scales are powers of two: dividing by them is exact, every code is one
// rounding (half to even) of the true quotient, and the matrix instructions
// apply them.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "flashopt.h"
#include "flashopt_fp8.h"
#include "flashopt_internal.h"

namespace flashopt {
namespace {

// -------------------------------------------------------------- quantize

// A tile of 128 x 128: both kinds of group, or a block, whole.  A wavefront
// takes 32 of the rows; a lane eight rows (8 (lane / 16) on) of eight columns
// (8 (lane % 16) on), so that a group along a row is sixteen lanes of one load,
// and eight rows of a column are eight bytes of its codes.
constexpr int kTile = 128, kLane = 8;

// The codes of a column's eight rows, in the order of the rows.
template <bool F32, int FMT>
__device__ __forceinline__ u32x2 column_codes(const Eight<F32> (&f)[kLane], int j, uint32_t scale)
{
    u32x2 q;
    if constexpr (F32) {
        q.x = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f[0].w[j], f[1].w[j], scale), f[2].w[j], f[3].w[j], scale);
        q.y = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f[4].w[j], f[5].w[j], scale), f[6].w[j], f[7].w[j], scale);
    } else {
        const int k = j >> 1;
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        auto pair = [&](int i) { return __builtin_amdgcn_perm(f[i + 1].w[k], f[i].w[k], sel); };
        q.x = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, pair(0), scale), pair(2), scale);
        q.y = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, pair(4), scale), pair(6), scale);
    }
    return q;
}

// What a norm multiplies its rows and columns by on the way to 8 bits.
struct NormFactors {
    const float *rstd;       // [rows]
    const uint8_t *gain;     // [cols] bf16 or fp32
    bool gain_fp32;
};

__device__ __forceinline__ Eight<true> gain8(const NormFactors &n, int64_t c, int64_t cols)
{
    if (n.gain_fp32) return load8<true, false>(n.gain + c * 4, cols - c);
    const Eight<false> g = load8<false, false>(n.gain + c * 2, cols - c);
    Eight<true> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.w[j] = __float_as_uint(value(g, j));
    return v;
}

// Codes of x along its rows (ROWS), of its transpose (COLS), or both, from one
// read; BLOCK: under one scale; NORM: of (x rstd) gain, each product rounded
// to fp32.  Codes along columns go through LDS to be stored in lines.  Bound by
// memory: 8192 x 5632 bf16 both ways 37 us (186 MB: 5.0 TB/s), along columns
// alone 28; 14336 x 4096 both ways in blocks 42 (235 MB: 5.6); 333 x 1001 fp32
// both ways 6.5, where 24 workgroups wait for their loads and stores in turn.
// A tile is what a column's scale needs, 128 rows, by one line of bytes.
template <bool F32, int FMT, bool ROWS, bool COLS, bool BLOCK, bool NORM>
__global__ void __launch_bounds__(kThreads)
fp8_quantize_kernel(const uint8_t *__restrict__ x, int64_t rows, int64_t cols, int64_t row_bytes,
                    uint32_t col_tiles, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                    uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t, NormFactors norm)
{
    constexpr bool W = F32 || NORM;          // the type that is quantized
    constexpr int kWaves = kThreads / kWaveLanes, kWords = W ? 8 : 4, kEsz = F32 ? 4 : 2;
    __shared__ __align__(16) u32x2 s_codes[COLS ? kTile * (kTile / kLane) : 1];
    __shared__ __align__(16) uint32_t s_top[COLS || BLOCK ? kWaves * 16 * kWords : 1];
    __shared__ uint8_t s_bytes[COLS ? kTile : 1];
    const int lane = threadIdx.x & (kWaveLanes - 1), l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const uint32_t tile = xcd_contiguous(blockIdx.x, gridDim.x);
    const int64_t tile_col = static_cast<int64_t>(tile % col_tiles) * kTile;
    const int64_t tile_row = static_cast<int64_t>(tile / col_tiles) * kTile;
    const int64_t row0 = tile_row + wave * 32 + q * kLane, c = tile_col + l16 * kLane;
    const bool inside = tile_col + kTile <= cols && tile_row + kTile <= rows;

    // rows past the end repeat the last and then count as zeros
    Eight<W> f[kLane];
    {
        Eight<F32> raw[kLane];
        auto row = [&](int i) { return x + (row0 + i < rows ? row0 + i : rows - 1) * row_bytes + c * kEsz; };
        if (inside) {
            const uint8_t *p = x + row0 * row_bytes + c * kEsz;
#pragma unroll
            for (int i = 0; i < kLane; ++i, p += row_bytes) raw[i] = load8<F32, !NORM>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kLane; ++i) raw[i] = load8<F32, !NORM>(row(i), cols - c);
        }
        if constexpr (NORM) {
            const Eight<true> g = gain8(norm, c, cols);
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                const float r = norm.rstd[row0 + i < rows ? row0 + i : rows - 1];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = (value(raw[i], j) * r) * value(g, j);
                    f[i].w[j] = inside || c + j < cols ? __float_as_uint(v) : 0u;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLane; ++i)
#pragma unroll
                for (int w = 0; w < kWords; ++w) f[i].w[w] = raw[i].w[w];
        }
        if (!inside) {
#pragma unroll
            for (int i = 0; i < kLane; ++i)
                if (row0 + i >= rows) f[i] = Eight<W>{};
        }
    }

    Eight<W> top{};
    if constexpr (COLS || BLOCK) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) raise(top, f[i]);
    }
    uint32_t block_top = 0u;
    if constexpr (BLOCK) {
        const uint32_t t = across16(max16(largest(top)), [](uint32_t a, uint32_t b) { return umax32(a, b); });
        if (lane == 0) s_top[wave] = t;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) block_top = umax32(block_top, s_top[w]);
    } else if constexpr (COLS) {
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            top.w[w] = across16(top.w[w], [](uint32_t a, uint32_t b) { return W ? umax32(a, b) : max_u16(a, b); });
        if (q == 0) {
#pragma unroll
            for (int w = 0; w < kWords; w += 4)
                *reinterpret_cast<u32x4 *>(&s_top[(wave * 16 + l16) * kWords + w]) =
                    u32x4{top.w[w], top.w[w + 1], top.w[w + 2], top.w[w + 3]};
        }
    }

    const int64_t colsp = mx_padded(cols), rowsp = mx_padded(rows);
    const int64_t col_scales = fp8_scale_stride(cols), row_scales = fp8_scale_stride(rows);
    if constexpr (ROWS) {
        uint32_t keep = 0u;                   // lane l16: the byte of row l16
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            const uint32_t t = BLOCK ? block_top : max16(largest_of(f[i]));
            const uint32_t scale = fp8_scale<FMT>(t);
            u32x2 codes8 = row_codes<W, FMT>(f[i], scale);
            uint32_t b = scale >> 23;
            if (t >= kInfinite) {
                codes8 = u32x2{0u, 0u};
                b = kNanByte;
            }
            keep = l16 == i ? b : keep;
            if (inside || row0 + i < rows) *reinterpret_cast<u32x2 *>(codes + (row0 + i) * colsp + c) = codes8;
        }
        if (l16 < kLane && row0 + l16 < rows) {
            uint8_t *p = scales + (row0 + l16) * col_scales + tile_col / kTile;
            *p = static_cast<uint8_t>(keep);
            if (tile_col + kTile >= cols)     // the rest of the padded row of scales
                for (int64_t i = 1; tile_col / kTile + i < col_scales; ++i) p[i] = 0;
        }
    }
    if constexpr (COLS) {
        if constexpr (!BLOCK) {
            __syncthreads();
            top = Eight<W>{};
#pragma unroll
            for (int v = 0; v < kWaves; ++v)
#pragma unroll
                for (int w = 0; w < kWords; w += 4) {
                    const u32x4 t = *reinterpret_cast<const u32x4 *>(&s_top[(v * 16 + l16) * kWords + w]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top.w[w + k] = W ? umax32(top.w[w + k], t[k]) : max_u16(top.w[w + k], t[k]);
                }
        }
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const uint32_t t = BLOCK ? block_top : __float_as_uint(value(top, j));
            const uint32_t scale = fp8_scale<FMT>(t);
            u32x2 codes8 = column_codes<W, FMT>(f, j, scale);
            uint32_t b = scale >> 23;
            if (t >= kInfinite) {
                codes8 = u32x2{0u, 0u};
                b = kNanByte;
            }
            // 8-byte slots, a column's sixteen turned by the lane so that
            // sixteen lanes' stores fall on all banks
            s_codes[(l16 * kLane + j) * 16 + ((wave * 4 + q) ^ l16)] = codes8;
            if (wave == 0 && q == 0) s_bytes[l16 * kLane + j] = static_cast<uint8_t>(b);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile * kTile / 16 / kThreads; ++i) {
            const int u = i * kThreads + threadIdx.x, col = u / 8, turn = (col / kLane) & 15;
            if (inside || tile_col + col < cols) {
                u32x4 v = *reinterpret_cast<const u32x4 *>(&s_codes[col * 16 + ((2 * (u % 8)) ^ (turn & 14))]);
                if (turn & 1) v = u32x4{v.z, v.w, v.x, v.y};
                *reinterpret_cast<u32x4 *>(codes_t + (tile_col + col) * rowsp + tile_row + (u % 8) * 16) = v;
            }
        }
        const int col = threadIdx.x;
        if (col < kTile && tile_col + col < cols) {
            uint8_t *p = scales_t + (tile_col + col) * row_scales + tile_row / kTile;
            *p = s_bytes[col];
            if (tile_row + kTile >= rows)
                for (int64_t i = 1; tile_row / kTile + i < row_scales; ++i) p[i] = 0;
        }
    }
}

// Codes along rows alone: a wavefront takes four groups of four rows, sixteen
// lanes to a group, and needs no LDS: 8192 x 5632 bf16 25 us (140 MB: 5.5 TB/s),
// 333 x 1001 fp32 3.2 (in tiles of 128 rows, as above, 5.0).
constexpr int kRowsAtOnce = 4;

template <bool F32, int FMT>
__global__ void __launch_bounds__(kThreads)
fp8_rows_kernel(const uint8_t *__restrict__ x, int64_t rows, int64_t cols, int64_t row_bytes,
                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int64_t colsp = mx_padded(cols), stride = fp8_scale_stride(cols);
    // below 2^24 tiles of 128 x 128 there are less than 2^32 items: 32-bit
    // division (with one of 64 bits 16 x 4096 takes 3.05 us for 2.8, 8192 x 4096 19 for 18)
    const uint32_t quads = static_cast<uint32_t>(stride / 4);
    const uint32_t total = static_cast<uint32_t>((rows + kRowsAtOnce - 1) / kRowsAtOnce) * quads;
    for (uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / kWaveLanes) + threadIdx.x / kWaveLanes);
         item < total; item += gridDim.x * (kThreads / kWaveLanes)) {
        const int64_t row0 = static_cast<int64_t>(item / quads) * kRowsAtOnce;
        const int64_t group = item % quads * 4 + (lane >> 4), c = group * 128 + (lane & 15) * 8;
        Eight<F32> f[kRowsAtOnce];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int64_t row = row0 + i < rows ? row0 + i : rows - 1;
            f[i] = load8<F32, true>(x + row * row_bytes + c * (F32 ? 4 : 2), cols - c);
        }
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const uint32_t top = max16(largest_of(f[i])), scale = fp8_scale<FMT>(top);
            u32x2 q = row_codes<F32, FMT>(f[i], scale);
            uint32_t b = scale >> 23;
            if (top >= kInfinite) {
                q = u32x2{0u, 0u};
                b = kNanByte;
            }
            if (row0 + i >= rows) break;
            if (c < colsp) *reinterpret_cast<u32x2 *>(codes + (row0 + i) * colsp + c) = q;
            if ((lane & 15) == 0) scales[(row0 + i) * stride + group] = static_cast<uint8_t>(b);
        }
    }
}

// ------------------------------------------------------------ dequantize

// The value of a scale byte: 2^(b - 127), subnormal at b = 0, NaN at 255.
__device__ __forceinline__ float scale_value(uint32_t b)
{
    if (b == 0u) return __uint_as_float(0x00400000u);
    return __uint_as_float(b == kNanByte ? 0x7FC00000u : b << 23);
}

// The four values of a word of codes.
template <int FMT>
__device__ __forceinline__ void values4(uint32_t w, float (&v)[4])
{
    f32x2 lo, hi;
    if constexpr (FMT == kE5M2) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, 1.0f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, 1.0f, true);
    } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, true);
    }
    v[0] = lo.x;
    v[1] = lo.y;
    v[2] = hi.x;
    v[3] = hi.y;
}

// One thread per eight columns; 14336 x 4096 to bf16 29-31 us (177 MB: 5.7-6.1
// TB/s).
template <bool F32, int FMT>
__global__ void __launch_bounds__(kThreads)
fp8_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                      int64_t cols, uint8_t *__restrict__ out, int64_t row_bytes)
{
    const int64_t colsp = mx_padded(cols), stride = fp8_scale_stride(cols), per_row = (cols + 7) / 8;
    const int64_t total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / per_row, c = (i - r * per_row) * 8;
        const u32x2 w = *reinterpret_cast<const u32x2 *>(codes + r * colsp + c);
        const float s = scale_value(scales[r * stride + c / 128]);
        float v[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float four[4];
            values4<FMT>(w[k], four);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * k + e] = four[e] * s;
        }
        store8<F32>(out + r * row_bytes + c * (F32 ? 4 : 2), rounded8<F32>(v), cols - c);
    }
}

// --------------------------------------------------------------- product

// out[m, n] = sum_k A[m, k] B[n, k].  The matrix instructions take rows of B
// as their first operand and rows of A as their second, so that a lane's
// accumulators hold consecutive n of one m, and stores run along out's rows.
// B is E4M3; A is either.

struct Fp8In {
    const uint8_t *codes, *scales;
    int64_t rows;
};

template <int FMT>
__device__ __forceinline__ f32x4 mfma16(i32x8 b, i32x8 a, f32x4 c, uint32_t sb, uint32_t sa)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, kE4M3, FMT, 0, static_cast<int>(sb), 0,
                                                            static_cast<int>(sa));
}

// One row of A: a plain sum of products, without the matrix instructions, so
// that a wavefront reads 1024 consecutive bytes of a row of B at a time, sixteen
// to a lane.  A workgroup takes two rows of B, its wavefronts take such pieces
// in turn and add their sums in order.  A lane's sixteen products are added in
// fp32 unscaled and then scaled by both scales' exponents together.
//
// Bound by memory: with the weight in cache / with weights in turn that no cache
// holds 14336 x 4096 takes 11.5 / 12.3 us (59 MB: 5.1 / 4.8 TB/s), 4096 x 14336
// 11.8 / 14.0, 4096 x 4096 4.5 / 5.9, 28672 x 8192 36.8 / 45.  (As a tile of 16
// rows of A by fp8_few_kernel: 12.4 / 17.2, 11.7 / 13.7, 5.0 / 7.0, 38 / 47; with
// one row to a wavefront, four or eight, or fewer wavefronts to a row, up to 20%
// slower.  Two rows of A are level with the tile.)
constexpr int kVectorRows = 2, kVectorWaves = kThreads / kWaveLanes;

// A as it is stored, or a row of bf16 that each workgroup quantizes for itself
// (as fp8_rows_kernel does, bit for bit): that saves a launch before this one.
template <int FMT>
struct StoredRow {
    static constexpr int kFormat = FMT;
    const uint8_t *codes, *scales;
    __device__ __forceinline__ u32x4 load(uint32_t at, bool there, uint32_t group, uint32_t &byte) const
    {
        byte = 0u;
        if (!there) return u32x4{0u, 0u, 0u, 0u};
        byte = scales[group];
        return *reinterpret_cast<const u32x4 *>(codes + at);
    }
};
struct RawRow {
    static constexpr int kFormat = kE4M3;
    const uint8_t *data;
    int64_t cols;
    __device__ __forceinline__ u32x4 load(uint32_t at, bool, uint32_t, uint32_t &byte) const
    {
        const uint8_t *p = data + at * 2u;
        const int count = static_cast<int>(cols) - static_cast<int>(at);
        const Eight<false> lo = load8<false, false>(p, count), hi = load8<false, false>(p + 16, count - 8);
        Eight<false> top{};
        raise(top, lo);
        raise(top, hi);
        uint32_t t = largest(top);               // over the eight lanes of a group
        t = umax32(t, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(t), 0xB1, 0xF, 0xF, true)));
        t = umax32(t, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(t), 0x4E, 0xF, 0xF, true)));
        t = umax32(t, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(t), 0x141, 0xF, 0xF, true)));
        const uint32_t scale = fp8_scale<kE4M3>(t);
        const u32x2 a = row_codes<false, kE4M3>(lo, scale), b = row_codes<false, kE4M3>(hi, scale);
        byte = t >= kInfinite ? kNanByte : scale >> 23;
        return t >= kInfinite ? u32x4{0u, 0u, 0u, 0u} : u32x4{a.x, a.y, b.x, b.y};
    }
};

template <typename A>
__global__ void __launch_bounds__(kThreads)
fp8_vector_kernel(A a, Fp8In b, int64_t kp, int64_t stride, uint8_t *__restrict__ out, bool out_fp32)
{
    constexpr int R = kVectorRows;
    __shared__ float s_sum[2][kVectorWaves][R];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int pieces = static_cast<int>((kp + 1023) / 1024), last = static_cast<int>(b.rows) - 1;
    const uint32_t groups = (static_cast<uint32_t>(b.rows) + R - 1) / R;
    int turn = 0;
    for (uint32_t group = blockIdx.x; group < groups; group += gridDim.x, turn ^= 1) {
        const uint8_t *codes[R], *scales[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = static_cast<int>(group * R) + r < last ? static_cast<int>(group * R) + r : last;
            codes[r] = b.codes + row * kp;
            scales[r] = b.scales + row * stride;
        }
        float acc[R] = {};
        // (unrolled twice, 30% slower where a wavefront has one piece)
#pragma unroll 1
        for (int c = wave; c < pieces; c += kVectorWaves) {
            const uint32_t at = static_cast<uint32_t>(c) * 1024u + lane * 16u, of = at / 128u;
            const bool there = at < static_cast<uint32_t>(kp);
            u32x4 wb[R];
            uint32_t eb[R], ea;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                wb[r] = u32x4{0u, 0u, 0u, 0u};
                eb[r] = 0u;
                if (there) {
                    wb[r] = *reinterpret_cast<const u32x4 *>(codes[r] + at);
                    eb[r] = scales[r][of];
                }
            }
            const u32x4 wa = a.load(at, there, of, ea);
            float part[R] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float va[4], vb[4];
                values4<A::kFormat>(wa[q], va);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    values4<kE4M3>(wb[r][q], vb);
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[r] = __builtin_fmaf(va[i], vb[i], part[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                acc[r] += ea == kNanByte || eb[r] == kNanByte
                              ? __uint_as_float(0x7FC00000u)
                              : __builtin_amdgcn_ldexpf(part[r], static_cast<int>(ea + eb[r]) - 254);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float x = wave_sum(acc[r]);
            if (lane == 0) s_sum[turn][wave][r] = x;
        }
        __syncthreads();
        const uint32_t n = group * R + threadIdx.x;
        if (threadIdx.x < R && n <= static_cast<uint32_t>(last)) {
            float x = s_sum[turn][0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kVectorWaves; ++w) x += s_sum[turn][w][threadIdx.x];
            if (out_fp32) reinterpret_cast<float *>(out)[n] = x;
            else reinterpret_cast<uint16_t *>(out)[n] = bf16_rne(x);
        }
    }
}

// Few rows of A, or few tiles: a workgroup takes 16 NT rows of B and 16 MT of A;
// its wavefronts take steps of 128 elements of K, four in succession, and add
// their sums at the end, in wavefront order.  Each copies its own steps to LDS
// of its own by the DMA, up to three ahead, and waits for nobody.  Scales go to
// LDS 128 steps at a time.  LDS holds rows as the tiles below do.
//
// What bounds it is how much a CU has under way: 48 x 4096 x 14336 takes 14.6 us
// with the weight in cache and 20-22 with weights in turn that no cache holds
// (59 MB: 4.0 and 2.8 TB/s), 16 x 14336 x 4096 12.7 and 18-19, 256 x 4096 x 14336
// 25.5 and 34.  (Loaded by the lanes that use them, operands take sixteen
// rows' half lines an instruction, where the copies take eight rows' whole
// ones, and the first of these 34 us, or 30 with four steps' loads at once.)
constexpr int kFewWaves = 4, kFewThreads = kFewWaves * kWaveLanes;

template <int MT, int NT>
struct Few {
    static constexpr int kRows = 16 * (MT + NT), kBytes = kRows * 128, kCopies = kRows / 8;
    static constexpr int kStages = kFewWaves * kBytes * 4 <= 144 * 1024 - kRows * 144 ? 4 : 2;
    static constexpr int kBlock = 128, kPitch = 144;       // steps whose scales LDS holds, and bytes of a row of them
};

template <int N>
__device__ __forceinline__ void wait_vm()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

template <int FMT, int MT, int NT>
__global__ void __launch_bounds__(kFewThreads)
fp8_few_kernel(Fp8In a, Fp8In b, int64_t kp, int64_t stride, uint8_t *__restrict__ out, bool out_fp32,
               int64_t row_bytes)
{
    using T = Few<MT, NT>;
    constexpr int kWaves = kFewWaves, kStages = T::kStages;
    __shared__ __align__(128) uint8_t s_buf[kWaves][kStages][T::kBytes];
    __shared__ __align__(16) uint8_t s_scales[T::kRows][T::kPitch];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t tiles_n = (b.rows + 16 * NT - 1) / (16 * NT), tiles_m = (a.rows + 16 * MT - 1) / (16 * MT);
    const int all_steps = static_cast<int>(kp / 128);
    const uint32_t chunk = ((lane & 7) ^ (lane >> 4)) * 16;   // of rows 0 to 7 of 16: bit 2 turned for the others
    const uint32_t lds_to = lds_offset(s_buf[wave]);
    for (int64_t tile = blockIdx.x; tile < tiles_n * tiles_m; tile += gridDim.x) {
        const int64_t n0 = tile % tiles_n * (16 * NT), m0 = tile / tiles_n * (16 * MT);
        const int n_last = static_cast<int>(b.rows - n0 < 16 * NT ? b.rows - n0 : 16 * NT) - 1;
        const int m_last = static_cast<int>(a.rows - m0 < 16 * MT ? a.rows - m0 : 16 * MT) - 1;
        // rows of B, then of A; past the end the last one again, unstored
        uint32_t src[T::kCopies];
#pragma unroll
        for (int i = 0; i < T::kCopies; ++i) {
            const int r = (i < 2 * NT ? i : i - 2 * NT) * 8 + (lane >> 3), last = i < 2 * NT ? n_last : m_last;
            src[i] = __umul24(r < last ? r : last, static_cast<uint32_t>(kp)) + (chunk ^ ((i & 1) * 64u));
        }
        const uint8_t *b_codes = b.codes + n0 * kp, *a_codes = a.codes + m0 * kp;
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int first = 0; first < all_steps; first += T::kBlock) {
            const int count = all_steps - first < T::kBlock ? all_steps - first : T::kBlock;
            // this wavefront's steps t = 0, 1, ...: fours of them in turn with the other wavefronts'
            const int fours = (count + 3) / 4, mine = (fours - wave + kWaves - 1) / kWaves;
            const int tail = mine > 0 && ((mine - 1) * kWaves + wave) * 4 + 4 > count ? 4 - (count & 3) : 0;
            const int steps = 4 * mine - tail;
            auto issue = [&](int t, int stage) {
                const int64_t at = static_cast<int64_t>(first + ((t >> 2) * kWaves + wave) * 4 + (t & 3)) * 128;
                const uint32_t to = lds_to + stage * T::kBytes;
#pragma unroll
                for (int i = 0; i < T::kCopies; ++i)
                    load_to_lds((i < 2 * NT ? b_codes : a_codes) + at, src[i], to + i * 1024);
            };
#pragma unroll
            for (int t = 0; t < kStages - 1; ++t)
                if (t < steps) issue(t, t);
            for (int u = threadIdx.x; u < T::kRows * 8; u += kFewThreads) {
                const int r = u >> 3, at = first + (u & 7) * 16;
                const bool of_b = r < 16 * NT;
                const int row = of_b ? r : r - 16 * NT, last = of_b ? n_last : m_last;
                const uint8_t *p = (of_b ? b.scales + n0 * stride : a.scales + m0 * stride) +
                                   static_cast<int64_t>(row < last ? row : last) * stride;
                if (at < stride)
                    *reinterpret_cast<u32x4 *>(&s_scales[r][(u & 7) * 16]) = *reinterpret_cast<const u32x4 *>(p + at);
            }
            __syncthreads();
            for (int q = 0; q < mine; ++q) {
                uint32_t sb[NT], sa[MT];
                const int word = (q * kWaves + wave) * 4;
#pragma unroll
                for (int i = 0; i < NT; ++i) sb[i] = *reinterpret_cast<const uint32_t *>(&s_scales[16 * i + l16][word]);
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    sa[j] = *reinterpret_cast<const uint32_t *>(&s_scales[16 * (NT + j) + l16][word]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = 4 * q + u, left = steps - 1 - t;
                    if (left < 0) break;
                    // the last step's reads are done: its buffer is the next copy's
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (left >= kStages - 1) {
                        issue(t + kStages - 1, (u + kStages - 1) % kStages);
                        wait_vm<(kStages - 1) * T::kCopies>();
                    } else if (left == 2) {
                        wait_vm<(kStages > 2 ? 2 : 0) * T::kCopies>();
                    } else if (left == 1) {
                        wait_vm<(kStages > 2 ? 1 : 0) * T::kCopies>();
                    } else {
                        wait_vm<0>();
                    }
                    const uint8_t *buf = s_buf[wave][u % kStages];
                    auto operand = [&](int tile16) {
                        const uint8_t *row = buf + tile16 * 2048 + l16 * 128;
                        const uint32_t x = (g ^ ((l16 >> 1) & 7)) * 16;
                        const u32x4 lo = *reinterpret_cast<const u32x4 *>(row + x);
                        const u32x4 hi = *reinterpret_cast<const u32x4 *>(row + (x ^ 64));
                        return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z),
                                     static_cast<int>(lo.w), static_cast<int>(hi.x), static_cast<int>(hi.y),
                                     static_cast<int>(hi.z), static_cast<int>(hi.w)};
                    };
                    i32x8 vb[NT], va[MT];
#pragma unroll
                    for (int i = 0; i < NT; ++i) vb[i] = operand(i);
#pragma unroll
                    for (int j = 0; j < MT; ++j) va[j] = operand(NT + j);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < MT; ++j)
                            acc[i][j] = mfma16<FMT>(vb[i], va[j], acc[i][j], sb[i] >> (8 * u), sa[j] >> (8 * u));
                }
            }
            __syncthreads();                     // every wavefront's reads of the scales and its copies are done
        }
        f32x4(*s_acc)[NT][MT][kWaveLanes] = reinterpret_cast<f32x4(*)[NT][MT][kWaveLanes]>(&s_buf[0][0][0]);
        static_assert(kWaves * NT * MT * kWaveLanes * 16 <= kWaves * kStages * T::kBytes, "sums");
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) s_acc[wave][i][j][lane] = acc[i][j];
        __syncthreads();
        for (int i = wave; i < NT * MT; i += kWaves) {
            f32x4 v = s_acc[0][i / MT][i % MT][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                const f32x4 u = s_acc[w][i / MT][i % MT][lane];
                v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            const int64_t m = m0 + 16 * (i % MT) + l16, n = n0 + 16 * (i / MT) + 4 * g;
            if (m >= a.rows) continue;
            if (out_fp32) store4<true>(out, row_bytes, m, n, b.rows, v.x, v.y, v.z, v.w);
            else store4<false>(out, row_bytes, m, n, b.rows, v.x, v.y, v.z, v.w);
        }
        __syncthreads();
    }
}

// A wavefront's turned-over rows of out: so many at a time.
__host__ __device__ constexpr int stage_rows(bool f32) { return f32 ? 8 : 16; }
__host__ __device__ constexpr int stage_bytes(bool f32, int tn) { return stage_rows(f32) * tn * 32 * (f32 ? 4 : 2); }

// Larger products: a workgroup computes a BN x BM tile of out^T, its
// wavefronts in a WN x WM arrangement of 32 x 32 accumulator blocks.
//
// Each K step is one group of 128 elements, one 128-byte line of every row,
// copied from global memory to LDS by the DMA (16 bytes to a lane, eight rows
// an instruction).  LDS holds row r's 16-byte chunk c at slot c ^ (r / 2 & 7)
// of the row's 128 bytes: the DMA writes lanes in order, so each lane fetches
// the chunk that belongs to its slot, and the 32 rows that an operand read
// takes at one c then fall on all banks.  Two buffers, and one barrier past the
// middle of a step: by then its buffer has been read, so the copy of the step
// after next goes there, and the next step's first operands are fetched, under
// the remaining products.
//
// A step is two products of 64 elements on each block.  They run along A's
// blocks, each with all of B's: a wavefront holds B's operands of both halves
// and a ring of A's, of eight registers each, which leaves room for 128
// accumulators among 256 registers.
//
// Scales: each thread carries 16 bytes of one row, sixteen steps' worth, through
// a register to LDS; a lane fetches a word, four steps' worth, of each of its
// rows and shifts it by a byte a step.
//
// What bounds it: 8192^3 takes 401-422 us (2.6-2.7 PFLOP/s) with random
// operands, 8192 x 14336 x 4096 365-399 (of fp32 outputs, twice their bytes, 438
// and 421), where the bare instruction on registers
// reaches 4.05 PFLOP/s (4.95 on zeros): the card's power.  The matrix units are
// busy 71% of the cycles (61% of the second's) at a clock that is held to 1.9
// GHz; without the copies, or without the reads of LDS, a copy of the kernel
// keeps the same cycles' share at 2.0 and 2.3 GHz, and without its stores the
// second takes 5% less.  Two groups of wavefronts in turn, one reading while the
// other multiplies, are busy 79% at 1.78 GHz and 3% faster on 8192^3, 5% slower
// over short K; four wavefronts of 128 x 128, a third fewer reads, 5% faster on
// 8192^3 and as much slower on 8192 x 14336 x 4096; workgroups that start one
// after another, so that their stores fall apart, 1% slower.
template <int BN, int BM, int WN, int WM>
struct Tile {
    static constexpr int kWaves = WN * WM;
    static constexpr int kTileThreads = kWaves * kWaveLanes;
    static constexpr int kRows = BN + BM;                  // rows of B, then of A
    static constexpr int kBytes = kRows * 128;             // one buffer
    // half of the wavefronts copy B, half A: DMA instructions of one and step
    static constexpr int kCopiesB = BN / 4 / kWaves, kCopiesA = BM / 4 / kWaves;
    static constexpr int kCopies = kCopiesB > kCopiesA ? kCopiesB : kCopiesA;
    static constexpr int kTN = BN / WN / 32, kTM = BM / WM / 32;
    static constexpr int kWavesPerSimd = BN * BM >= 128 * 128 ? 2 : 4;
    // A's operands of a step in their order, the ring that holds them, and how
    // far ahead of its products one is fetched
    static constexpr int kSeq = 2 * kTM, kRing = kSeq < 4 ? kSeq : kSeq % 4 == 0 ? 4 : 3, kAhead = kRing - 1;
    static constexpr int kLds(bool f32) { return 2 * kBytes + 2 * kRows * 16 + kWaves * stage_bytes(f32, kTN); }
    static_assert(BN % (4 * kWaves) == 0 && BM % (4 * kWaves) == 0 && BN % (32 * WN) == 0 && BM % (32 * WM) == 0 &&
                      kSeq % kRing == 0 && kRows <= kTileThreads && BN % kWaveLanes == 0, "tile");
};

template <bool F32, int FMT, int BN, int BM, int WN, int WM>
__global__ void __launch_bounds__(WN *WM *kWaveLanes)
    __attribute__((amdgpu_waves_per_eu(Tile<BN, BM, WN, WM>::kWavesPerSimd)))
fp8_tile_kernel(Fp8In a, Fp8In b, int64_t kp, int64_t stride, uint32_t tiles_n, uint32_t tiles_m,
                uint8_t *__restrict__ out, int64_t row_bytes)
{
    using T = Tile<BN, BM, WN, WM>;
    constexpr int kTN = T::kTN, kTM = T::kTM;
    __shared__ __align__(128) uint8_t s_buf[2][T::kBytes];
    __shared__ uint32_t s_scales[2][4][T::kRows];
    __shared__ __align__(16) uint8_t s_stage[T::kWaves][stage_bytes(F32, kTN)];
    const int thread = threadIdx.x, lane = thread & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(thread / kWaveLanes);
    const int wn = wave % WN, wm = wave / WN, g = lane >> 5;
    const uint32_t code_stride = static_cast<uint32_t>(kp), scale_stride = static_cast<uint32_t>(stride);
    const int steps = static_cast<int>(kp / 128);
    const uint32_t total = tiles_n * tiles_m;

    // The copies run two steps ahead of the products, through the tiles in
    // turn: tile pt, step pk is copied next.  A wavefront copies rows of one
    // matrix only, and thread t the scales of buffer row t: uniform bases, and
    // 32-bit offsets of the lane, row x stride (24 bits each, kp being below
    // 2^24).  Rows are clamped to the matrix: a row past the end repeats the
    // last one, unstored.
    uint32_t pt = blockIdx.x;
    int pk = 0;
    const bool copy_b = wave < T::kWaves / 2, scale_b = wave * kWaveLanes < BN;
    const int first_copy = copy_b ? wave * T::kCopiesB : (wave - T::kWaves / 2) * T::kCopiesA;
    const uint8_t *copy_base = nullptr, *scale_base = nullptr;
    uint32_t src[T::kCopies], scale_src = 0;
    // slot s of row r holds chunk s ^ ((r / 2) & 7): for rows 0 to 7 of 16
    // here, for rows 8 to 15 with bit 2 of the chunk turned
    const uint32_t chunk = ((lane & 7) ^ (lane >> 4)) * 16;
    auto aim = [&] {
        uint32_t tile_n, tile_m;
        tile_at(pt, tiles_n, tiles_m, tile_n, tile_m);
        const int64_t n0 = static_cast<int64_t>(tile_n) * BN, m0 = static_cast<int64_t>(tile_m) * BM;
        const int n_last = static_cast<int>(b.rows - n0 < BN ? b.rows - n0 : BN) - 1;
        const int m_last = static_cast<int>(a.rows - m0 < BM ? a.rows - m0 : BM) - 1;
        copy_base = copy_b ? b.codes + n0 * code_stride : a.codes + m0 * code_stride;
        scale_base = scale_b ? b.scales + n0 * scale_stride : a.scales + m0 * scale_stride;
        const int copy_last = copy_b ? n_last : m_last, scale_last = scale_b ? n_last : m_last;
        const int first = first_copy * 8 + (lane >> 3);
#pragma unroll
        for (int i = 0; i < T::kCopies; ++i) {
            const int r = first + 8 * i;
            src[i] = __umul24(r < copy_last ? r : copy_last, code_stride) + (chunk ^ ((i & 1) * 64u));
        }
        const int r = thread - (scale_b ? 0 : BN);
        scale_src = __umul24(r < scale_last ? r : scale_last, scale_stride);
    };
    const uint32_t lds_to = lds_offset(s_buf) + (copy_b ? 0 : BN * 128) + first_copy * 1024;
    auto copy = [&](int i, int buf) {
        if (i >= T::kCopiesB && copy_b) return;
        if (i >= T::kCopiesA && !copy_b) return;
        load_to_lds(copy_base, src[i], lds_to + buf * T::kBytes + i * 1024);
    };

    // Quarter q of a lane's row: its chunk 2 q + g; a product takes two.
    const uint32_t off = (lane & 31) * 128 + ((g ^ ((lane >> 1) & 7)) << 4);
    auto operand = [&](int buf, int half, int row) {
        const uint8_t *p = &s_buf[buf][row * 128];
        const u32x4 x = *reinterpret_cast<const u32x4 *>(p + (off ^ (64 * half)));
        const u32x4 y = *reinterpret_cast<const u32x4 *>(p + (off ^ (64 * half + 32)));
        return i32x8{static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w),
                     static_cast<int>(y.x), static_cast<int>(y.y), static_cast<int>(y.z), static_cast<int>(y.w)};
    };
    i32x8 vn[2][kTN], vm[T::kRing];
    auto fetch_n = [&](int buf, int half, int i) { vn[half][i] = operand(buf, half, (wn * kTN + i) * 32); };
    auto fetch_m = [&](int buf, int s) {
        vm[s % T::kRing] = operand(buf, s / kTM, BN + (wm * kTM + s % kTM) * 32);
    };

    f32x16 acc[kTN][kTM];
    uint32_t word_n[kTN], word_m[kTM];           // four steps' scales of a row

    // After the copies of step pk: with the first of sixteen steps, their
    // scales go to a register, and before the next barrier settle() moves them
    // to LDS.  Past the last tile its last copies are repeated, unused.
    u32x4 next_scales{0u, 0u, 0u, 0u};
    bool pending = false;
    int pset = 1, set = 0;       // sets of scales: the last one filled, the one in use
    auto advance = [&] {
        if (!(pk & 15)) {
            pset ^= 1;
            if (T::kRows == T::kTileThreads || thread < T::kRows)
                next_scales = *reinterpret_cast<const u32x4 *>(scale_base + scale_src + pk);
            pending = true;
        }
        copy_base += 128;
        if (++pk == steps) {
            if (pt + gridDim.x < total) {
                pk = 0;
                pt += gridDim.x;
                aim();
            } else {
                --pk;
                copy_base -= 128;
            }
        }
    };
    auto settle = [&] {
        if (!pending) return;
        if (T::kRows == T::kTileThreads || thread < T::kRows) {
#pragma unroll
            for (int w = 0; w < 4; ++w) s_scales[pset][w][thread] = next_scales[w];
        }
        pending = false;
    };
    auto fetch_scales = [&](int k) {
        const uint32_t *from = s_scales[set][(k >> 2) & 3] + (lane & 31);
#pragma unroll
        for (int i = 0; i < kTN; ++i) word_n[i] = from[(wn * kTN + i) * 32];
#pragma unroll
        for (int i = 0; i < kTM; ++i) word_m[i] = from[BN + (wm * kTM + i) * 32];
    };

    uint32_t t = blockIdx.x;
    if (t >= total) return;
    aim();
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) copy(i, 0);
    advance();
    __builtin_amdgcn_s_waitcnt(0);       // this wavefront's copies have reached LDS
    settle();
    __syncthreads();                     // everyone's have
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) copy(i, 1);
    advance();
#pragma unroll
    for (int i = 0; i < kTN; ++i) fetch_n(0, 0, i);
#pragma unroll
    for (int s = 0; s < T::kAhead; ++s) fetch_m(0, s);
    fetch_scales(0);
    int buf = 0;
    for (; t < total; t += gridDim.x) {
#pragma unroll
        for (int i = 0; i < kTN; ++i)
#pragma unroll
            for (int j = 0; j < kTM; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        for (int k = 0; k < steps; ++k, buf ^= 1) {
            const bool last = k == steps - 1;
            // Product x: A's operand s with B's block i.  Each is pinned in its
            // place, with the reads of LDS and copies that go before it.
            constexpr int kSwap = T::kSeq - T::kAhead;     // the operand before which the buffers change
#pragma unroll
            for (int x = 0; x < T::kSeq * kTN; ++x) {
                const int s = x / kTN, i = x % kTN, half = s / kTM, j = s % kTM;
                if (s < kSwap) {
                    if (i == 0) fetch_m(buf, s + T::kAhead);
                    // B's second half, as soon as that leaves room
                    if (x < kTN) fetch_n(buf, 1, x);
                }
                if (x == kSwap * kTN) {
                    __builtin_amdgcn_s_waitcnt(0);
                    settle();
                    __syncthreads();
                    if ((k & 15) == 15 || last) set ^= 1;
                }
                if (s >= kSwap) {
                    const int y = x - kSwap * kTN, left = (T::kSeq - kSwap) * kTN;
                    // the next step's first operands: B's once the first half's
                    // products are done, A's as the ring frees them
                    const int z = x - (kSwap > kTM ? kSwap : kTM) * kTN;
                    if (z >= 0 && z < kTN) fetch_n(buf ^ 1, 0, z);
                    if (i == 0 && s > kSwap) fetch_m(buf ^ 1, s - kSwap - 1);
                    const int per = (T::kCopies + left - 1) / left;
#pragma unroll
                    for (int c = y * per; c < (y + 1) * per && c < T::kCopies; ++c) copy(c, buf);
                }
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    vn[half][i], vm[s % T::kRing], acc[i][j], kE4M3, FMT, 0, static_cast<int>(word_n[i]), 0,
                    static_cast<int>(word_m[j]));
                asm volatile("" : "+v"(acc[i][j]));
                __builtin_amdgcn_sched_barrier(0);
            }
            if ((k & 3) == 3 || last) {
                fetch_scales(last ? 0 : k + 1);
            } else {
#pragma unroll
                for (int i = 0; i < kTN; ++i) word_n[i] >>= 8;
#pragma unroll
                for (int i = 0; i < kTM; ++i) word_m[i] >>= 8;
            }
            fetch_m(buf ^ 1, T::kAhead - 1);
            advance();
        }
        // Block element e of a lane is m = lane % 32, n = 8 (e / 4) +
        // 4 (lane / 32) + e % 4: 16 bytes of a row at most, where a store of
        // part of a line costs L2 as much as one of a whole line.  Each
        // wavefront turns a few rows at a time over in LDS of its own and
        // stores them in 16-byte pieces, whole lines of bf16; the next tile's
        // copies run meanwhile.  (As a function of its own this takes 1-2%
        // more of the whole kernel's time.)
        constexpr int kEsz = F32 ? 4 : 2, kPitch = kTN * 32 * kEsz, kR = stage_rows(F32), kPieces = kPitch / 16;
        uint32_t tile_n, tile_m;
        tile_at(t, tiles_n, tiles_m, tile_n, tile_m);
        const int64_t m_first = static_cast<int64_t>(tile_m) * BM + wm * (kTM * 32);
        const int64_t n_first = static_cast<int64_t>(tile_n) * BN + wn * (kTN * 32);
        uint8_t *stage = s_stage[wave];
        // where piece c of row r lies in the row, so that 16 rows' pieces c
        // fall on all banks
        auto turned = [](int r, int c) { return (c ^ ((r * kPieces / 16) & (kPieces - 1))) * 16; };
#pragma unroll
        for (int j = 0; j < kTM; ++j) {
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += kR) {
                if ((lane & (32 - kR)) == r0) {
#pragma unroll
                    for (int i = 0; i < kTN; ++i)
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const f32x16 &x = acc[i][j];
                            const int r = lane & (kR - 1), n = i * 32 + 2 * e + 4 * g;
                            uint8_t *p = stage + r * kPitch + turned(r, n * kEsz / 16) + n * kEsz % 16;
                            if constexpr (F32)
                                *reinterpret_cast<f32x4 *>(p) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
                            else
                                *reinterpret_cast<u32x2 *>(p) =
                                    u32x2{bf16_pair(x[e], x[e + 1]), bf16_pair(x[e + 2], x[e + 3])};
                        }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int u0 = 0; u0 < kR * kPieces; u0 += kWaveLanes) {
                    const int u = u0 + lane, r = u / kPieces, c = u % kPieces;
                    const int64_t m = m_first + j * 32 + r0 + r, n = n_first + c * (16 / kEsz);
                    if (u < kR * kPieces && m < a.rows && n < b.rows) {
                        const u32x4 w = *reinterpret_cast<const u32x4 *>(stage + r * kPitch + turned(r, c));
                        uint8_t *o = out + m * row_bytes + n * kEsz;
                        if (n + 16 / kEsz <= b.rows) {
                            *reinterpret_cast<u32x4_packed *>(o) = w;
                        } else {
#pragma unroll
                            for (int x = 0; x < 16 / kEsz; ++x) {
                                if (n + x >= b.rows) break;
                                if constexpr (F32) reinterpret_cast<uint32_t *>(o)[x] = w[x];
                                else
                                    reinterpret_cast<uint16_t *>(o)[x] =
                                        static_cast<uint16_t>(w[x / 2] >> (16 * (x & 1)));
                            }
                        }
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0);       // no copy outlives the workgroup's LDS
}

// ------------------------------------------------------------- launching

template <bool F32, int FMT, bool BLOCK, bool NORM>
hipError_t quantize_tiles(const MxMatrix &x, const Fp8Out &q, const NormFactors &norm, hipStream_t st)
{
    const uint32_t col_tiles = static_cast<uint32_t>((x.cols + kTile - 1) / kTile);
    const uint32_t row_tiles = static_cast<uint32_t>((x.rows + kTile - 1) / kTile);
    const dim3 grid(col_tiles * row_tiles), block(kThreads);
    const int64_t row_bytes = x.row_stride * (F32 ? 4 : 2);
    const uint8_t *p = static_cast<const uint8_t *>(x.data);
    if (q.codes && q.codes_t)
        hipLaunchKernelGGL((fp8_quantize_kernel<F32, FMT, true, true, BLOCK, NORM>), grid, block, 0, st, p, x.rows,
                           x.cols, row_bytes, col_tiles, q.codes, q.scales, q.codes_t, q.scales_t, norm);
    else if (q.codes_t)
        hipLaunchKernelGGL((fp8_quantize_kernel<F32, FMT, false, true, BLOCK, NORM>), grid, block, 0, st, p, x.rows,
                           x.cols, row_bytes, col_tiles, q.codes, q.scales, q.codes_t, q.scales_t, norm);
    else if constexpr (BLOCK)
        hipLaunchKernelGGL((fp8_quantize_kernel<F32, FMT, true, false, BLOCK, NORM>), grid, block, 0, st, p, x.rows,
                           x.cols, row_bytes, col_tiles, q.codes, q.scales, q.codes_t, q.scales_t, norm);
    return hipGetLastError();
}

template <bool F32, int FMT>
hipError_t quantize_type(const MxMatrix &x, bool block, const Fp8Out &q, hipStream_t st)
{
    if (block) return quantize_tiles<F32, FMT, true, false>(x, q, NormFactors{}, st);
    if (q.codes_t) return quantize_tiles<F32, FMT, false, false>(x, q, NormFactors{}, st);
    const int64_t waves = (x.rows + kRowsAtOnce - 1) / kRowsAtOnce * (fp8_scale_stride(x.cols) / 4);
    const int64_t blocks = (waves + kThreads / kWaveLanes - 1) / (kThreads / kWaveLanes);
    hipLaunchKernelGGL((fp8_rows_kernel<F32, FMT>), dim3(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20))),
                       dim3(kThreads), 0, st, static_cast<const uint8_t *>(x.data), x.rows, x.cols,
                       x.row_stride * (F32 ? 4 : 2), q.codes, q.scales);
    return hipGetLastError();
}

template <typename A>
hipError_t vector(const A &a, const Fp8In &b, int64_t k, uint8_t *out, bool out_fp32, hipStream_t st)
{
    const int64_t groups = (b.rows + kVectorRows - 1) / kVectorRows;
    hipLaunchKernelGGL((fp8_vector_kernel<A>), dim3(static_cast<unsigned>(groups < (1 << 20) ? groups : (1 << 20))),
                       dim3(kThreads), 0, st, a, b, mx_padded(k), fp8_scale_stride(k), out, out_fp32);
    return hipGetLastError();
}

int64_t few_tiles(const Fp8In &a, const Fp8In &b, int mt, int nt)
{
    return ((a.rows + 16 * mt - 1) / (16 * mt)) * ((b.rows + 16 * nt - 1) / (16 * nt));
}

template <int FMT, int MT, int NT>
hipError_t few(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, bool out_fp32, int64_t row_bytes,
               hipStream_t st)
{
    const int64_t tiles = few_tiles(a, b, MT, NT);
    const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
    hipLaunchKernelGGL((fp8_few_kernel<FMT, MT, NT>), dim3(grid), dim3(kFewThreads), 0, st, a, b, mx_padded(k),
                       fp8_scale_stride(k), out, out_fp32, row_bytes);
    return hipGetLastError();
}

template <bool F32, int FMT, int BN, int BM, int WN, int WM>
hipError_t tiles(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const uint32_t tn = static_cast<uint32_t>((b.rows + BN - 1) / BN);
    const uint32_t tm = static_cast<uint32_t>((a.rows + BM - 1) / BM);
    const uint64_t total = static_cast<uint64_t>(tn) * tm;
    if (total > UINT32_MAX / 2) return hipErrorInvalidValue;
    // as many workgroups as run at once (their LDS decides), each taking tiles
    // in turn; a multiple of the 8 XCDs
    constexpr unsigned kAtOnce = kCus * static_cast<unsigned>(160 * 1024 / Tile<BN, BM, WN, WM>::kLds(F32));
    const unsigned grid = total < kAtOnce ? static_cast<unsigned>(total) : kAtOnce;
    hipLaunchKernelGGL((fp8_tile_kernel<F32, FMT, BN, BM, WN, WM>), dim3(grid), dim3(WN * WM * kWaveLanes), 0, st, a,
                       b, mx_padded(k), fp8_scale_stride(k), tn, tm, out, row_bytes);
    return hipGetLastError();
}

// Elements of K from which 64 x 64 tiles, one or less to a CU, go to
// fp8_few_kernel, whose wavefronts split K, instead of fp8_tile_kernel.  M x N x
// K in us, by its tiles / by fp8_few_kernel: 1024 x 1000 x 1000 5.9 / 7.2, 200 x
// 4096 x 2048 7.8 / 7.7, 512 x 2048 x 2048 7.9 / 7.8, 256 x 4096 x 4096 12.4 / 11.2,
// 256 x 4096 x 14336 55.5 / 26.
constexpr int64_t kFewInner = 2048;

template <int FMT>
hipError_t product_format(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, bool out_fp32, int64_t row_bytes,
                          hipStream_t st)
{
    if (a.rows == 1) return vector(StoredRow<FMT>{a.codes, a.scales}, b, k, out, out_fp32, st);
    // The smallest tiles of which a CU gets one at most: a larger one reads A and
    // B less often, a smaller one leaves fewer CUs idle.  M x N x K in us, tiles
    // of 16 MT x 16 NT: 48 x 4096 x 14336 2 x 2 (256 tiles) 14.6, 3 x 2 17.4, 2 x 4
    // 18.4, 2 x 1 22.6; 48 x 14336 x 4096 3 x 4 (224) 14.5, 3 x 2 19.8, 2 x 2 27.9;
    // 24 x 6144 x 4096 2 x 2 (192) 7.0, 2 x 1 10.1; 64 x 2048 x 5632 2 x 1 (256)
    // 6.5, 2 x 2 6.8, 4 x 1 7.5; 128 x 4096 x 14336 4 x 2 (256) 20.7, 4 x 4 25.2, 2
    // x 2 27.5.
    const int64_t m16 = (a.rows + 15) / 16;
    auto fits = [&](int mt, int nt) { return mt <= m16 && few_tiles(a, b, mt, nt) <= kCus; };
    if (fits(1, 1)) return few<FMT, 1, 1>(a, b, k, out, out_fp32, row_bytes, st);
    if (fits(2, 1)) return few<FMT, 2, 1>(a, b, k, out, out_fp32, row_bytes, st);
    if (m16 == 1 && fits(1, 2)) return few<FMT, 1, 2>(a, b, k, out, out_fp32, row_bytes, st);
    if (fits(2, 2)) return few<FMT, 2, 2>(a, b, k, out, out_fp32, row_bytes, st);
    // One tile of A's rows, and B of more rows than that: 16 x 14336 x 4096 1 x 4
    // (224) 12.7, 1 x 1 15.1; 16 x 28672 x 8192 1 x 4 (448) 39.8, 1 x 1 (several to a
    // CU at once) 38.4, from memory 60.9 and 55.1; 32 x 28672 x 8192 2 x 4 41.5, 2 x 1
    // 53.0; 64 x 14336 x 4096 4 x 4 15.3, 64 x 64 tiles below 19.2.
    if (m16 == 1)
        return fits(1, 4) ? few<FMT, 1, 4>(a, b, k, out, out_fp32, row_bytes, st)
                          : few<FMT, 1, 1>(a, b, k, out, out_fp32, row_bytes, st);
    if (m16 == 3 && fits(3, 2)) return few<FMT, 3, 2>(a, b, k, out, out_fp32, row_bytes, st);
    if (m16 == 2) return few<FMT, 2, 4>(a, b, k, out, out_fp32, row_bytes, st);
    if (fits(4, 2)) return few<FMT, 4, 2>(a, b, k, out, out_fp32, row_bytes, st);
    if (m16 == 3) return few<FMT, 3, 4>(a, b, k, out, out_fp32, row_bytes, st);
    if (m16 == 4 || (fits(4, 4) && k >= kFewInner)) return few<FMT, 4, 4>(a, b, k, out, out_fp32, row_bytes, st);
    // The largest tile of which 160 are there for the 256 CUs: it reads A and B the
    // least often.  M x N x K in us, tiles of 256 / 128: 2048 x 4096 x 4096 (128 of
    // 256) 50.7 / 35.9, 2048 x 5120 x 4096 (160) 48.1 / 50.3, 2048 x 5120 x 1024 18.5 /
    // 18.5, 3328 x 3328 x 4096 (169) 48.7 / 51.3; tiles of 128 / 64: 1024 x 2048 x 2048
    // (128 of 128) 11.6 / 9.3, 1280 x 2048 x 2048 (160) 12.3 / 12.1, 1024 x 3328 x
    // 1000 (208) 8.9 / 10.3, 2048 x 2048 x 2048 (256) 13.3 / 16.7.
    const int64_t big = ((a.rows + 255) / 256) * ((b.rows + 255) / 256);
    const int64_t mid = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    // Of the two largest, 256 x 192 where that takes less of the turns that the
    // CUs take together, by three quarters of the work a turn.  256 x 256 / 256 x
    // 192: 5632 x 2048 x 8192 (176 tiles, 240) 90 / 80, 3328 x 3328 x 4096 (169, 234)
    // 48.7 / 43.7, 2560 x 4096 x 4096 (160, 224) 47.5 / 42.2, 2048 x 5120 x 1024 (160,
    // 220) 18.5 / 16.4, 4096 x 4608 x 4096 (288, 396) 94 / 78, 5632 x 6144 x 2048 (528,
    // 720) 79 / 70.  With fewer tiles, 128 x 128 are ahead: 2048 x 4096 x 4096 (128,
    // 176) 35.9 against 40.6.
    const int64_t low = ((a.rows + 191) / 192) * ((b.rows + 255) / 256);
    const bool lower = (low + kCus - 1) / kCus * 3 < (big + kCus - 1) / kCus * 4;
    auto in_tiles = [&](auto fp32) {
        constexpr bool F32 = decltype(fp32)::value;
        if (big >= 160 && lower) return tiles<F32, FMT, 256, 192, 4, 2>(a, b, k, out, row_bytes, st);
        if (big >= 160) return tiles<F32, FMT, 256, 256, 4, 2>(a, b, k, out, row_bytes, st);
        if (mid >= 160) return tiles<F32, FMT, 128, 128, 2, 2>(a, b, k, out, row_bytes, st);
        return tiles<F32, FMT, 64, 64, 2, 2>(a, b, k, out, row_bytes, st);
    };
    return out_fp32 ? in_tiles(std::true_type{}) : in_tiles(std::false_type{});
}

}  // namespace

hipError_t launch_fp8_quantize(const MxMatrix &x, int format, bool block, const Fp8Out &q, hipStream_t st)
{
    if (format == kE5M2)
        return x.fp32 ? quantize_type<true, kE5M2>(x, block, q, st) : quantize_type<false, kE5M2>(x, block, q, st);
    return x.fp32 ? quantize_type<true, kE4M3>(x, block, q, st) : quantize_type<false, kE4M3>(x, block, q, st);
}

hipError_t launch_fp8_normed(const MxMatrix &h, const float *rstd, const void *gain, bool gain_fp32, int format,
                             const Fp8Out &q, hipStream_t st)
{
    const NormFactors norm{rstd, static_cast<const uint8_t *>(gain), gain_fp32};
    if (format == kE5M2)
        return h.fp32 ? quantize_tiles<true, kE5M2, false, true>(h, q, norm, st)
                      : quantize_tiles<false, kE5M2, false, true>(h, q, norm, st);
    return h.fp32 ? quantize_tiles<true, kE4M3, false, true>(h, q, norm, st)
                  : quantize_tiles<false, kE4M3, false, true>(h, q, norm, st);
}

hipError_t launch_fp8_dequantize(const uint8_t *codes, const uint8_t *scales, int format, const MxMatrix &out,
                                 hipStream_t st)
{
    const int64_t threads = out.rows * ((out.cols + 7) / 8), blocks = (threads + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
    uint8_t *p = static_cast<uint8_t *>(out.data);
    const int64_t row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, codes, scales, out.rows, out.cols, p, row_bytes);
        return hipGetLastError();
    };
    if (format == kE5M2)
        return out.fp32 ? launch(fp8_dequantize_kernel<true, kE5M2>) : launch(fp8_dequantize_kernel<false, kE5M2>);
    return out.fp32 ? launch(fp8_dequantize_kernel<true, kE4M3>) : launch(fp8_dequantize_kernel<false, kE4M3>);
}

hipError_t launch_fp8_product(const uint8_t *a_codes, const uint8_t *a_scales, int a_format, const uint8_t *b_codes,
                              const uint8_t *b_scales, int64_t inner, const MxMatrix &out, hipStream_t st)
{
    const Fp8In a{a_codes, a_scales, out.rows}, b{b_codes, b_scales, out.cols};
    const int64_t row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    uint8_t *p = static_cast<uint8_t *>(out.data);
    if (inner == 0) {
        const int64_t blocks = (out.rows * out.cols + kThreads - 1) / kThreads;
        const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
        if (out.fp32) hipLaunchKernelGGL(zero_kernel<true>, grid, dim3(kThreads), 0, st, out.rows, out.cols, p, row_bytes);
        else hipLaunchKernelGGL(zero_kernel<false>, grid, dim3(kThreads), 0, st, out.rows, out.cols, p, row_bytes);
        return hipGetLastError();
    }
    return a_format == kE5M2 ? product_format<kE5M2>(a, b, inner, p, out.fp32, row_bytes, st)
                             : product_format<kE4M3>(a, b, inner, p, out.fp32, row_bytes, st);
}

bool fp8_linear_direct(const MxMatrix &x) { return x.rows == 1 && !x.fp32 && x.cols > 0; }

hipError_t launch_fp8_linear_direct(const MxMatrix &x, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const MxMatrix &out, hipStream_t st)
{
    return vector(RawRow{static_cast<const uint8_t *>(x.data), x.cols}, Fp8In{w_codes, w_scales, out.cols}, x.cols,
                  static_cast<uint8_t *>(out.data), out.fp32, st);
}

}  // namespace flashopt
