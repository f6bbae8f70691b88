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
// What bounds it: 8192^3 takes 408 us (2.7 PFLOP/s) with random operands, where
// the bare instruction on registers reaches 4.05 (4.95 on zeros): the card's
// power.  The matrix units are busy 71% of the cycles at a clock that is held
// to 1.9 GHz; without the copies, or without the reads of LDS, a copy of the
// kernel keeps the same cycles' share at 2.0 and 2.3 GHz.  Two groups of
// wavefronts in turn, one reading while the other multiplies, are busy 79% at
// 1.78 GHz and 3% faster on 8192^3, 5% slower over short K; four wavefronts of
// 128 x 128, a third fewer reads, 5% faster on 8192^3 and as much slower on
// 8192 x 14336 x 4096.
template <int BN, int BM, int WN, int WM>
struct Tile {
    static constexpr int kWaves = WN * WM;
    static constexpr int kTileThreads = kWaves * kWaveLanes;
    static constexpr int kRows = BN + BM;                  // rows of B, then of A
    static constexpr int kBytes = kRows * 128;             // one buffer
    static constexpr int kCopies = kRows / 8 / kWaves;     // DMA instructions of a wavefront and step
    static constexpr int kTN = BN / WN / 32, kTM = BM / WM / 32;
    static constexpr int kWavesPerSimd = BN * BM >= 128 * 128 ? 2 : 4;
    // A's operands of a step in their order, the ring that holds them, and how
    // far ahead of its products one is fetched
    static constexpr int kSeq = 2 * kTM, kRing = kSeq < 4 ? kSeq : 4, kAhead = kRing - 1;
    static constexpr int kLds(bool f32) { return 2 * kBytes + 2 * kRows * 16 + kWaves * stage_bytes(f32, kTN); }
    static_assert(kRows % (8 * kWaves) == 0 && BN % (32 * WN) == 0 && BM % (32 * WM) == 0 && kSeq % kRing == 0 &&
                      kRows <= kTileThreads && BN % (8 * kCopies) == 0 && BN % kWaveLanes == 0, "tile");
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
    const bool copy_b = wave * (8 * T::kCopies) < BN, scale_b = wave * kWaveLanes < BN;
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
        const int first = wave * (8 * T::kCopies) - (copy_b ? 0 : BN) + (lane >> 3);
#pragma unroll
        for (int i = 0; i < T::kCopies; ++i) {
            const int r = first + 8 * i;
            src[i] = __umul24(r < copy_last ? r : copy_last, code_stride) + (chunk ^ ((i & 1) * 64u));
        }
        const int r = thread - (scale_b ? 0 : BN);
        scale_src = __umul24(r < scale_last ? r : scale_last, scale_stride);
    };
    const uint32_t lds_to = lds_offset(s_buf) + wave * (T::kCopies * 1024);
    auto copy = [&](int i, int buf) { load_to_lds(copy_base, src[i], lds_to + buf * T::kBytes + i * 1024); };

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

template <bool F32, int FMT, int MT, int NT>
hipError_t skinny(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const int64_t tiles = ((b.rows + 16 * NT - 1) / (16 * NT)) * ((a.rows + 16 * MT - 1) / (16 * MT));
    const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
    hipLaunchKernelGGL((fp8_skinny_kernel<F32, FMT, MT, NT>), dim3(grid), dim3(kSkinnyWaves * kWaveLanes), 0, st, a,
                       b, mx_padded(k), fp8_scale_stride(k), out, row_bytes);
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

template <bool F32, int FMT>
hipError_t product_type(const Fp8In &a, const Fp8In &b, int64_t k, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    if (a.rows <= 16) return skinny<F32, FMT, 1, 1>(a, b, k, out, row_bytes, st);
    const int64_t m32 = (a.rows + 31) / 32;
    if (m32 * ((b.rows + 15) / 16) <= kCus) return skinny<F32, FMT, 2, 1>(a, b, k, out, row_bytes, st);
    if (m32 * ((b.rows + 31) / 32) <= kCus) return skinny<F32, FMT, 2, 2>(a, b, k, out, row_bytes, st);
    const int64_t big = ((a.rows + 255) / 256) * ((b.rows + 255) / 256);
    const int64_t mid = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    if (big >= 160) return tiles<F32, FMT, 256, 256, 4, 2>(a, b, k, out, row_bytes, st);
    if (mid >= 160) return tiles<F32, FMT, 128, 128, 2, 2>(a, b, k, out, row_bytes, st);
    return tiles<F32, FMT, 64, 64, 2, 2>(a, b, k, out, row_bytes, st);
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
