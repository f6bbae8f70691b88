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
// to fp32.  Codes along columns go through LDS to be stored in lines.
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
// lanes to a group, and needs no LDS.
constexpr int kRowsAtOnce = 4;

template <bool F32, int FMT>
__global__ void __launch_bounds__(kThreads)
fp8_rows_kernel(const uint8_t *__restrict__ x, int64_t rows, int64_t cols, int64_t row_bytes,
                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int64_t colsp = mx_padded(cols), stride = fp8_scale_stride(cols), quads = stride / 4;
    const int64_t total = (rows + kRowsAtOnce - 1) / kRowsAtOnce * quads;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / kWaveLanes) + threadIdx.x / kWaveLanes;
         item < total; item += static_cast<int64_t>(gridDim.x) * (kThreads / kWaveLanes)) {
        const int64_t row0 = item / quads * kRowsAtOnce;
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

// One thread per eight columns.
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
            f32x2 lo, hi;
            if constexpr (FMT == kE5M2) {
                lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w[k], 1.0f, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w[k], 1.0f, true);
            } else {
                lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[k], 1.0f, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[k], 1.0f, true);
            }
            v[4 * k] = lo.x * s;
            v[4 * k + 1] = lo.y * s;
            v[4 * k + 2] = hi.x * s;
            v[4 * k + 3] = hi.y * s;
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

__device__ __forceinline__ i32x8 load32(const uint8_t *p)
{
    const u32x4 a = *reinterpret_cast<const u32x4 *>(p), b = *reinterpret_cast<const u32x4 *>(p + 16);
    return i32x8{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
                 static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}

// Few rows of A: the time is B's, read once, so nothing is staged.  A workgroup
// takes 16 NT rows of B and 16 MT of A; its wavefronts take groups of 128
// elements of K in turn and add their sums at the end, in wavefront order.
// Within a step a lane holds 32 consecutive bytes of its row; any assignment of
// them to the instruction's K slots is the same sum, the scale being the
// row's for the whole step.
constexpr int kSkinnyWaves = 8;

template <bool F32, int FMT, int MT, int NT>
__global__ void __launch_bounds__(kSkinnyWaves *kWaveLanes)
fp8_skinny_kernel(Fp8In a, Fp8In b, int64_t kp, int64_t stride, uint8_t *__restrict__ out, int64_t row_bytes)
{
    __shared__ f32x4 s_acc[kSkinnyWaves][NT][MT][kWaveLanes];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t tiles_n = (b.rows + 16 * NT - 1) / (16 * NT), tiles_m = (a.rows + 16 * MT - 1) / (16 * MT);
    const int steps = static_cast<int>(kp / 128);
    for (int64_t tile = blockIdx.x; tile < tiles_n * tiles_m; tile += gridDim.x) {
        const int64_t n0 = tile % tiles_n * (16 * NT), m0 = tile / tiles_n * (16 * MT);
        const uint8_t *bp[NT], *bs[NT], *ap[MT], *as[MT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int64_t r = n0 + 16 * t + l16;
            if (r >= b.rows) r = b.rows - 1;     // read, never stored
            bp[t] = b.codes + r * kp + g * 32;
            bs[t] = b.scales + r * stride;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            int64_t r = m0 + 16 * t + l16;
            if (r >= a.rows) r = a.rows - 1;
            ap[t] = a.codes + r * kp + g * 32;
            as[t] = a.scales + r * stride;
        }
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = wave; k < steps; k += kSkinnyWaves) {
            i32x8 vb[NT], va[MT];
            uint32_t sb[NT], sa[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                vb[i] = load32(bp[i] + static_cast<int64_t>(k) * 128);
                sb[i] = bs[i][k];
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                va[j] = load32(ap[j] + static_cast<int64_t>(k) * 128);
                sa[j] = as[j][k];
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = mfma16<FMT>(vb[i], va[j], acc[i][j], sb[i], sa[j]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) s_acc[wave][i][j][lane] = acc[i][j];
        __syncthreads();
        for (int i = wave; i < NT * MT; i += kSkinnyWaves) {
            f32x4 v = s_acc[0][i / MT][i % MT][lane];
#pragma unroll
            for (int w = 1; w < kSkinnyWaves; ++w) {
                const f32x4 u = s_acc[w][i / MT][i % MT][lane];
                v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            const int64_t m = m0 + 16 * (i % MT) + l16, n = n0 + 16 * (i / MT) + 4 * g;
            if (m < a.rows) store4<F32>(out, row_bytes, m, n, b.rows, v.x, v.y, v.z, v.w);
        }
        __syncthreads();
    }
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

template <bool F32, int FMT, int MT, int NT>
hipError_t skinny(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const int64_t tiles = ((b.rows + 16 * NT - 1) / (16 * NT)) * ((a.rows + 16 * MT - 1) / (16 * MT));
    const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
    hipLaunchKernelGGL((fp8_skinny_kernel<F32, FMT, MT, NT>), dim3(grid), dim3(kSkinnyWaves * kWaveLanes), 0, st, a,
                       b, mx_padded(k), fp8_scale_stride(k), out, row_bytes);
    return hipGetLastError();
}

template <bool F32, int FMT>
hipError_t product_type(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    if (a.rows <= 16) return skinny<F32, FMT, 1, 1>(a, b, k, out, row_bytes, st);
    return skinny<F32, FMT, 2, 4>(a, b, k, out, row_bytes, st);
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
    if (a_format == kE5M2)
        return out.fp32 ? product_type<true, kE5M2>(a, b, inner, p, row_bytes, st)
                        : product_type<false, kE5M2>(a, b, inner, p, row_bytes, st);
    return out.fp32 ? product_type<true, kE4M3>(a, b, inner, p, row_bytes, st)
                    : product_type<false, kE4M3>(a, b, inner, p, row_bytes, st);
}

}  // namespace flashopt
