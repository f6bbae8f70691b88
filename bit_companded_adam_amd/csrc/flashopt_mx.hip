// MXFP4: E2M1 codes with one E8M0 scale for each 32 elements along a row
// (flashopt_mx_quantize, flashopt_mx_dequantize), and the product of two such
// matrices (flashopt_mx_product, flashopt_mx_linear).
//
// Storage of an R x C matrix: each row is padded to Cp = 128 ceil(C / 128)
// elements, so that a row's codes are whole 64-byte blocks, one K step of a
// matrix instruction, and its scales whole words; the product then has no
// ragged end along K.  codes: R rows of Cp / 2 bytes, the even column in the
// low nibble; scales: R rows of Cp / 32 bytes.  Padding is zero.
//
// Quantization of a group: with E the biased exponent of its largest
// magnitude, the scale is 2^(E - 127 - 2), so the largest value lands in
// [4, 8), the top binade of E2M1 (0 .5 1 1.5 2 3 4 6) and what saturates
// there.  The stored byte is max(E - 2, 0): scales below 2^-127 do not
// exist.  Dividing by the scale is exact, so every code is one rounding (half
// to even) of the true quotient.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "flashopt.h"
#include "flashopt_device.h"
#include "flashopt_internal.h"

namespace flashopt {
namespace {

// -------------------------------------------------------------- quantize

// Group maxima are kept as bit patterns without their sign, whose order is
// that of the magnitudes, infinities and NaN on top.  The scale 2^e as an fp32
// pattern is the maximum's exponent field less two, not below zero: the
// conversion instructions take their scale from the exponent field alone, so
// field 0 is 2^-127.
constexpr uint32_t kExponent = 0x7F800000u;
__device__ __forceinline__ uint32_t scale_bits(uint32_t top)
{
    return __builtin_elementwise_sub_sat(top & kExponent, 2u << 23);
}

// Maxima over aligned groups of eight lanes, of four rows at once: lane ^ 1,
// lane ^ 2, then the other four of the eight.  A DPP read needs two wait
// states after the write of its source, which the other three rows fill.
__device__ __forceinline__ void max8(uint32_t (&x)[4])
{
    asm("s_nop 1\n\t"
        "v_max_u32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %1, %1, %1 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %2, %2, %2 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %3, %3, %3 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %1, %1, %1 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %2, %2, %2 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %3, %3, %3 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %1, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_max_u32_dpp %3, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xf"
        : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]));
}

// Two E2M1 codes in byte SEL of acc (half to even, saturating at 6), from
// fp32 values or from a word of two bf16 ones.
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t acc, uint32_t a, uint32_t b, uint32_t scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(acc, __uint_as_float(a), __uint_as_float(b),
                                                    __uint_as_float(scale), SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t acc, uint32_t ab, uint32_t scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(acc, __builtin_bit_cast(bf16x2, ab),
                                                     __uint_as_float(scale), SEL);
}

// A wavefront takes 256 columns, four to a lane, of 32 rows, or of 8 where no
// groups along columns are wanted: every load covers 512 (bf16) or 1024 bytes
// of a row, a group along a row is eight lanes, and a group along a column is
// one lane's 32 values.
constexpr int kLaneCols = 4;
constexpr int kTileCols = 64 * kLaneCols;
constexpr int kQuantWaves = kThreads / kWaveLanes;
constexpr int quant_rows(bool columns) { return (columns ? 32 : 8) * kQuantWaves; }

// A lane's four values of one row, in the words they came in.
template <bool F32>
struct Four {
    uint32_t w[F32 ? 4 : 2];
};

template <bool F32>
__device__ __forceinline__ Four<F32> load4(const uint8_t *p)
{
    Four<F32> f;
    if constexpr (F32) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_packed *>(p));
        f.w[0] = v.x; f.w[1] = v.y; f.w[2] = v.z; f.w[3] = v.w;
    } else {
        const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_packed *>(p));
        f.w[0] = v.x; f.w[1] = v.y;
    }
    return f;
}
// One of the four, where the row ends within them.
template <bool F32>
__device__ __forceinline__ void load1(Four<F32> &f, int j, const uint8_t *p)
{
    if constexpr (F32) f.w[j] = *reinterpret_cast<const uint32_t *>(p + j * 4);
    else f.w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p + j * 2)) << (16 * (j & 1));
}

// Magnitude patterns: word by word, and the largest of the four as fp32 bits
// (for bf16 the low half holds other bits, which no use of it sees).
template <bool F32>
__device__ __forceinline__ Four<F32> magnitudes(const Four<F32> &f)
{
    Four<F32> m;
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) m.w[i] = f.w[i] & (F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
    return m;
}
template <bool F32>
__device__ __forceinline__ void raise(Four<F32> &a, const Four<F32> &b)
{
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) a.w[i] = F32 ? umax32(a.w[i], b.w[i]) : max_u16(a.w[i], b.w[i]);
}
template <bool F32>
__device__ __forceinline__ uint32_t largest(const Four<F32> &m)
{
    if constexpr (F32) return umax32(umax32(m.w[0], m.w[1]), umax32(m.w[2], m.w[3]));
    const uint32_t t = max_u16(m.w[0], m.w[1]);
    return umax32(t, t << 16);
}

// The codes of a column's eight consecutive rows, in the order of the rows.
template <bool F32>
__device__ __forceinline__ uint32_t column_codes(const Four<F32> *f, int j, uint32_t scale)
{
    if constexpr (F32) {
        uint32_t q = codes2<0>(0u, f[0].w[j], f[1].w[j], scale);
        q = codes2<1>(q, f[2].w[j], f[3].w[j], scale);
        q = codes2<2>(q, f[4].w[j], f[5].w[j], scale);
        return codes2<3>(q, f[6].w[j], f[7].w[j], scale);
    } else {
        const int k = j >> 1;
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        uint32_t q = codes2<0>(0u, __builtin_amdgcn_perm(f[1].w[k], f[0].w[k], sel), scale);
        q = codes2<1>(q, __builtin_amdgcn_perm(f[3].w[k], f[2].w[k], sel), scale);
        q = codes2<2>(q, __builtin_amdgcn_perm(f[5].w[k], f[4].w[k], sel), scale);
        return codes2<3>(q, __builtin_amdgcn_perm(f[7].w[k], f[6].w[k], sel), scale);
    }
}

// Codes of x along its rows (ROWS) and of its transpose (COLS), from one
// read.  Bound by memory: 8192 x 4096 takes 16.5 us along rows (85 MB, 5.2
// TB/s), 24 both ways (103 MB, 4.3 TB/s).  (Nontemporal stores save 2% and
// cost 1-6% with the product that reads the codes.)  With COLS a workgroup's four wavefronts take 128 rows, so that it
// writes 64 bytes of each column's codes and one word of its scales; those,
// and the rows', go through LDS to be stored in such pieces.
template <bool F32, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kThreads)
mx_quantize_kernel(const uint8_t *__restrict__ x, int64_t rows, int64_t cols, int64_t row_bytes,
                   uint32_t row_tiles, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t)
{
    constexpr int kTileRows = quant_rows(COLS), kWaveRows = kTileRows / kQuantWaves;
    __shared__ __align__(16) u32x4 s_codes[COLS ? kTileCols * kQuantWaves : 1];
    __shared__ __align__(16) uint8_t s_scales_t[COLS ? kTileCols * kQuantWaves : 1];
    __shared__ __align__(16) uint16_t s_rows[ROWS ? kTileRows * 64 : 1];
    __shared__ __align__(16) uint8_t s_scales[ROWS ? kTileRows * (kTileCols / 32) : 1];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    // the tiles of one XCD are neighbours down the rows: two of them write
    // the two halves of a line of codes_t
    const uint32_t tile = xcd_contiguous(blockIdx.x, gridDim.x);
    const int64_t tile_row = static_cast<int64_t>(tile % row_tiles) * kTileRows;
    const int64_t tile_col = static_cast<int64_t>(tile / row_tiles) * kTileCols;
    const int64_t row0 = tile_row + wave * kWaveRows, c = tile_col + lane * kLaneCols;
    const int64_t colsp = mx_padded(cols), rowsp = mx_padded(rows);

    Four<F32> f[kWaveRows];
    if (tile_col + kTileCols <= cols && row0 + kWaveRows <= rows) {
        const uint8_t *p = x + row0 * row_bytes + tile_col * (F32 ? 4 : 2);
        const uint32_t at = lane * (kLaneCols * (F32 ? 4 : 2));
#pragma unroll
        for (int r = 0; r < kWaveRows; ++r, p += row_bytes) f[r] = load4<F32>(p + at);
    } else {
        // rows past the end repeat the last and then count as zeros: no
        // branch, and so no wait, between the loads (1111 x 1000 bf16 both
        // ways: 11.2 us with one a row, 7.3 without)
        auto row = [&](int r) {
            return x + (row0 + r < rows ? row0 + r : rows - 1) * row_bytes + c * (F32 ? 4 : 2);
        };
#pragma unroll
        for (int r = 0; r < kWaveRows; ++r) f[r] = Four<F32>{};
        if (c + 4 <= cols) {
#pragma unroll
            for (int r = 0; r < kWaveRows; ++r) f[r] = load4<F32>(row(r));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < cols) {
#pragma unroll
                    for (int r = 0; r < kWaveRows; ++r) load1<F32>(f[r], j, row(r));
                }
        }
#pragma unroll
        for (int r = 0; r < kWaveRows; ++r)
            if (row0 + r >= rows) f[r] = Four<F32>{};
    }
    Four<F32> col_top{};
#pragma unroll
    for (int r = 0; r < kWaveRows; ++r) raise(col_top, magnitudes(f[r]));
    // infinities and NaN are rare: the selects for them run only where the
    // wavefront has seen one
    const bool bad = __any(largest(col_top) >= kExponent);

    if constexpr (ROWS) {
        // opaque, or the magnitudes above would be kept for the rows' maxima
        // and double the registers
#pragma unroll
        for (int r = 0; r < kWaveRows; ++r)
#pragma unroll
            for (int w = 0; w < (F32 ? 4 : 2); ++w) asm volatile("" : "+v"(f[r].w[w]));
        uint32_t keep[kWaveRows / 8] = {};       // lane l: the scale of its group in rows l % 8 + 8 i
        auto four_rows = [&](int r0, auto check) {
            uint32_t top[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = largest(magnitudes(f[r0 + i]));
            max8(top);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + i;
                const uint32_t scale = scale_bits(top[i]);
                uint32_t q, b = scale >> 23;
                if constexpr (F32) {
                    q = codes2<0>(0u, f[r].w[0], f[r].w[1], scale);
                    q = codes2<1>(q, f[r].w[2], f[r].w[3], scale);
                } else {
                    q = codes2<0>(0u, f[r].w[0], scale);
                    q = codes2<1>(q, f[r].w[1], scale);
                }
                if (decltype(check)::value && top[i] >= kExponent) {
                    q = 0u;
                    b = 255u;
                }
                keep[r / 8] = (lane & 7) == (r & 7) ? b : keep[r / 8];
                s_rows[(wave * kWaveRows + r) * 64 + lane] = static_cast<uint16_t>(q);
            }
            __builtin_amdgcn_sched_barrier(0);   // a few rows at a time: fewer registers, more wavefronts
        };
        if (!bad) {
#pragma unroll
            for (int r = 0; r < kWaveRows; r += 4) four_rows(r, std::false_type{});
        } else {
#pragma unroll
            for (int r = 0; r < kWaveRows; r += 4) four_rows(r, std::true_type{});
        }
#pragma unroll
        for (int i = 0; i < kWaveRows / 8; ++i)
            s_scales[(wave * kWaveRows + 8 * i + (lane & 7)) * (kTileCols / 32) + lane / 8] =
                static_cast<uint8_t>(keep[i]);
    }
    if constexpr (COLS) {
#pragma unroll
        for (int j = 0; j < kLaneCols; ++j) {
            uint32_t top;
            if constexpr (F32) top = col_top.w[j];
            else top = (j & 1) ? col_top.w[j / 2] & 0xFFFF0000u : col_top.w[j / 2] << 16;
            const uint32_t scale = scale_bits(top);
            uint32_t b = scale >> 23;
            u32x4 q{column_codes(&f[0], j, scale), column_codes(&f[8], j, scale), column_codes(&f[16], j, scale),
                    column_codes(&f[24], j, scale)};
            if (bad && top >= kExponent) {
                q = u32x4{0u, 0u, 0u, 0u};
                b = 255u;
            }
            const int col = lane * kLaneCols + j;
            // 16-byte slots, the eight that share the banks turned by the
            // lane so that eight lanes' stores fall on all of them
            s_codes[(col * kQuantWaves + wave) ^ (lane & 7)] = q;
            s_scales_t[col * kQuantWaves + wave] = static_cast<uint8_t>(b);
        }
    }
    __syncthreads();
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < kTileRows * 8 / kThreads; ++i) {
            const int u = i * kThreads + threadIdx.x;
            const int64_t row = tile_row + u / 8, byte = tile_col / 2 + (u % 8) * 16;
            if (row < rows && byte < colsp / 2)
                *reinterpret_cast<u32x4 *>(codes + row * (colsp / 2) + byte) =
                    *reinterpret_cast<const u32x4 *>(&s_rows[u * 8]);
        }
        const int r = threadIdx.x;                // eight groups to a row of the tile, fours of them there or not
        if (r < kTileRows && tile_row + r < rows) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(&s_scales[r * (kTileCols / 32)]);
            uint8_t *p = scales + (tile_row + r) * (colsp / 32) + tile_col / 32;
            *reinterpret_cast<uint32_t *>(p) = v.x;
            if (tile_col + 128 < colsp) *reinterpret_cast<uint32_t *>(p + 4) = v.y;
        }
    }
    if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < kQuantWaves; ++i) {
            const int u = i * kThreads + threadIdx.x, col = u / kQuantWaves;
            if (tile_col + col < cols)
                *reinterpret_cast<u32x4 *>(codes_t + (tile_col + col) * (rowsp / 2) + tile_row / 2 +
                                           (u % kQuantWaves) * 16) = s_codes[u ^ ((col / kLaneCols) & 7)];
        }
        const int col = threadIdx.x;
        if (tile_col + col < cols)
            *reinterpret_cast<uint32_t *>(scales_t + (tile_col + col) * (rowsp / 32) + tile_row / 32) =
                *reinterpret_cast<const uint32_t *>(&s_scales_t[col * kQuantWaves]);
    }
}

// ------------------------------------------------------------ dequantize

// The value of a scale byte: 2^(b - 127), subnormal at b = 0, NaN at 255.
__device__ __forceinline__ float scale_value(uint32_t b)
{
    if (b == 0u) return __uint_as_float(0x00400000u);
    return __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);
}

// One thread per eight columns.  8192 x 4096 takes 15.3 us to bf16 and 25.5 to
// fp32 (85 and 152 MB: 5.6 and 6.0 TB/s).  (Nontemporal stores save 4 us and
// cost the next reader of out 5.)
template <bool F32>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                     int64_t cols, uint8_t *__restrict__ out, int64_t row_bytes)
{
    const int64_t colsp = mx_padded(cols), per_row = (cols + 7) / 8, total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / per_row, c = (i - r * per_row) * 8;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + r * (colsp / 2) + c / 2);
        const float s = scale_value(scales[r * (colsp / 32) + c / 32]);
        float v[8];
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
        v[4] = d.x * s; v[5] = d.y * s; v[6] = e.x * s; v[7] = e.y * s;
        uint8_t *o = out + r * row_bytes;
        if (c + 8 <= cols) {
            u32x4 p;
            if constexpr (F32) {
                for (int k = 0; k < 4; ++k) p[k] = __float_as_uint(v[k]);
                *reinterpret_cast<u32x4_packed *>(o + c * 4) = p;
                for (int k = 0; k < 4; ++k) p[k] = __float_as_uint(v[4 + k]);
                *reinterpret_cast<u32x4_packed *>(o + c * 4 + 16) = p;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
                *reinterpret_cast<u32x4_packed *>(o + c * 2) = p;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c + k >= cols) break;
                if constexpr (F32) reinterpret_cast<float *>(o)[c + k] = v[k];
                else reinterpret_cast<uint16_t *>(o)[c + k] = bf16_rne(v[k]);
            }
        }
    }
}

// --------------------------------------------------------------- product

// out[m, n] = sum_k A[m, k] B[n, k].  The matrix instructions take rows of B
// as their first operand and rows of A as their second, so that a lane's
// accumulators hold consecutive n of one m, and stores run along out's rows.

struct MxIn {
    const uint8_t *codes, *scales;
    int64_t rows;
};

__device__ __forceinline__ i32x8 operand(u32x4 v)
{
    return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z),
                 static_cast<int>(v.w), 0, 0, 0, 0};
}

template <int BYTE>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(a), operand(b), c, 4, 4, BYTE, static_cast<int>(sa), BYTE, static_cast<int>(sb));
}

template <int BYTE>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        operand(a), operand(b), c, 4, 4, BYTE, static_cast<int>(sa), BYTE, static_cast<int>(sb));
}

// Few rows of A: the time is B's, read once, so nothing is staged.  A workgroup
// takes 16 NT rows of B and 16 MT of A; its wavefronts take 256-element steps
// of K in turn and add their sums at the end, in wavefront order.
// Within a step a lane holds groups 2 g and 2 g + 1 of its row (g = lane / 16):
// 32 consecutive bytes, and any assignment of groups to the instruction's
// four K slots is the same sum as long as both operands and their scales
// agree.  Eight wavefronts, so that 4096 rows of B still fill the chip.  With
// the weight in cache from the call before / with weights in turn that no cache
// holds, 1 x 4096 x 4096 takes 3.6 / 5.0 us (8.9 MB), 1 x 14336 x 4096 8.4 / 9.4
// (31 MB, 3.7 / 3.3 TB/s), 1 x 28672 x 8192 26.5 / 28.1 (125 MB, 4.7 / 4.5 TB/s):
// latency, of the launch, one pass over K and the sum across wavefronts.  (Two
// steps' loads ahead are level; nontemporal ones, or 64 contiguous bytes of a
// row in each, 10-20% slower.)
constexpr int kSkinnyWaves = 8;

struct Step {
    u32x4 lo, hi;
    uint32_t scale;      // byte 0: lo's, byte 1: hi's
};

__device__ __forceinline__ Step load_step(const MxIn &in, int64_t row, int64_t kp, int64_t group)
{
    Step s{u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}, 0u};
    if (group < kp / 32) {            // groups come in fours: both are there, or neither
        const uint8_t *p = in.codes + row * (kp / 2) + group * 16;
        s.lo = *reinterpret_cast<const u32x4 *>(p);
        s.hi = *reinterpret_cast<const u32x4 *>(p + 16);
        s.scale = *reinterpret_cast<const uint16_t *>(in.scales + row * (kp / 32) + group);
    }
    return s;
}

// A's rows as they come, in bf16, 16-byte aligned and of whole 16-byte pieces:
// a lane's two groups are 64 elements of its own, so they are quantized where
// they are used (as mx_quantize_kernel does, bit for bit).  Every workgroup
// does it again: worth it while A is a few rows.
struct MxRaw {
    const uint8_t *data;
    int64_t rows, row_bytes, cols;
};

// The codes of the 32 elements at p, of which `count` exist, and their scale.
__device__ __forceinline__ u32x4 quantize_group(const uint8_t *p, int64_t count, uint32_t &byte)
{
    u32x4 w[4], q;
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = u32x4{0u, 0u, 0u, 0u};
        if (i * 8 < count) w[i] = *reinterpret_cast<const u32x4 *>(p + i * 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) top = max_u16(top, w[i][x] & 0x7FFF7FFFu);
    top = umax32(top, top << 16);
    const uint32_t scale = scale_bits(top);
    byte = scale >> 23;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c = codes2<0>(0u, w[i].x, scale);
        c = codes2<1>(c, w[i].y, scale);
        c = codes2<2>(c, w[i].z, scale);
        q[i] = codes2<3>(c, w[i].w, scale);
    }
    if (top >= kExponent) {
        byte = 255u;
        q = u32x4{0u, 0u, 0u, 0u};
    }
    return q;
}

__device__ __forceinline__ Step load_step(const MxRaw &in, int64_t row, int64_t, int64_t group)
{
    const int64_t first = group * 32;
    const uint8_t *p = in.data + row * in.row_bytes + first * 2;
    uint32_t lo, hi;
    Step s;
    s.lo = quantize_group(p, in.cols - first, lo);
    s.hi = quantize_group(p + 64, in.cols - first - 32, hi);
    s.scale = lo | (hi << 8);
    return s;
}

template <bool F32, int MT, int NT, typename A>
__global__ void __launch_bounds__(kSkinnyWaves *kWaveLanes)
mx_skinny_kernel(A a, MxIn b, int64_t kp, uint8_t *__restrict__ out, int64_t row_bytes)
{
    __shared__ f32x4 s_acc[kSkinnyWaves][NT][MT][kWaveLanes];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t tiles = (b.rows + 16 * NT - 1) / (16 * NT);
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
    const int steps = static_cast<int>((kp + 255) / 256);
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t n0 = tile * (16 * NT);
        int64_t brow[NT], arow[MT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            brow[t] = n0 + 16 * t + l16;
            if (brow[t] >= b.rows) brow[t] = b.rows - 1;     // read, never stored
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            arow[t] = m0 + 16 * t + l16;
            if (arow[t] >= a.rows) arow[t] = a.rows - 1;
        }
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = wave; k < steps; k += kSkinnyWaves) {
            const int64_t group = static_cast<int64_t>(k) * 8 + 2 * g;
            Step sb[NT], sa[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) sb[i] = load_step(b, brow[i], kp, group);
#pragma unroll
            for (int j = 0; j < MT; ++j) sa[j] = load_step(a, arow[j], kp, group);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    acc[i][j] = mfma16<0>(sb[i].lo, sa[j].lo, acc[i][j], sb[i].scale, sa[j].scale);
                    acc[i][j] = mfma16<1>(sb[i].hi, sa[j].hi, acc[i][j], sb[i].scale, sa[j].scale);
                }
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

// Larger products: a workgroup computes a BN x BM tile of out^T, its
// wavefronts in a WN x WM arrangement of 32 x 32 accumulator blocks; with KS
// > 1 that many such groups take a share of K each, and the first adds the
// shares' sums in their order.
//
// Each K step of 256 elements is 128 bytes of every row, one cache line,
// copied from global memory to LDS by the DMA (16 bytes to a lane, eight rows
// an instruction).  LDS holds row r's 16-byte chunk c at slot c ^ (r / 2 & 7)
// of the row's 128 bytes: the DMA writes lanes in order, so each lane fetches
// the chunk that belongs to its slot, and the 32 rows that an operand read
// takes at one c then fall on all banks.  Two buffers, and one barrier near
// the end of a step: by then its buffer has been read, so the copy of the step
// after next goes there and has a whole step's products to land in.
//
// Scales: each thread carries 16 bytes of one row, two steps' worth, through
// a register to LDS.  (Loaded by the lanes that use them they cost 32 cache
// lines an instruction, and set the time: 8192^3 took 485 us.)  The four that
// a lane needs of a step's eight (groups 2 k + lane / 32) are gathered into
// one word with a byte permutation, and the instruction selects its byte.
//
// What bounds it: 8192^3 takes 256-261 us (4.2-4.3 PFLOP/s) on random codes
// and 190 us (5.8) on zeros, where the bare instructions on registers reach 6.4
// and 9.1 PFLOP/s, 172 and 121 us: random operands cost clock, the rest is
// waiting for copies and about 5 us a tile for storing out, while every CU
// stores.  Four wavefronts of 128 x 128 instead of eight of 64 x 128 (a third
// fewer LDS reads, accumulators in AGPRs) take 275 us: nothing runs beside a
// wavefront's own waits then.
template <int BN, int BM, int WN, int WM>
struct Tile {
    static constexpr int kWaves = WN * WM;
    static constexpr int kTileThreads = kWaves * kWaveLanes;
    static constexpr int kRows = BN + BM;                  // rows of B, then of A
    static constexpr int kBytes = kRows * 128;             // one buffer
    static constexpr int kCopies = kRows / 8 / kWaves;     // DMA instructions of a wavefront and step
    static constexpr int kTN = BN / WN / 32, kTM = BM / WM / 32;
    // as LDS allows; the compiler keeps accumulators out of the AGPRs (moves
    // around each pinned product) where it is held to this
    static constexpr int kWavesPerSimd = BN * BM >= 128 * 128 ? 2 : 4;
    // a wavefront's turned-over rows of out: so many at a time
    static constexpr int kStageRows(bool f32) { return f32 ? 8 : 16; }
    static constexpr int kPitch(bool f32) { return kTN * 32 * (f32 ? 4 : 2); }
    static constexpr int kLds(bool f32)
    {
        return 2 * kBytes + 2 * kRows * 16 + kWaves * kStageRows(f32) * kPitch(f32);
    }
    static_assert(kRows % (8 * kWaves) == 0 && BN % (32 * WN) == 0 && BM % (32 * WM) == 0 &&
                      kRows <= kTileThreads && BN % (8 * kCopies) == 0 && BN % kWaveLanes == 0, "tile");
};

template <bool F32, int BN, int BM, int WN, int WM, int KS>
__global__ void __launch_bounds__(KS *WN *WM *kWaveLanes)
    __attribute__((amdgpu_waves_per_eu(Tile<BN, BM, WN, WM>::kWavesPerSimd)))
mx_tile_kernel(MxIn a, MxIn b, int64_t kp, uint32_t tiles_n, uint32_t tiles_m, uint8_t *__restrict__ out,
               int64_t row_bytes)
{
    using T = Tile<BN, BM, WN, WM>;
    constexpr int kTN = T::kTN, kTM = T::kTM;
    __shared__ __align__(128) uint8_t s_bufs[KS][2][T::kBytes];
    __shared__ u32x4 s_scale_sets[KS][2][T::kRows];
    __shared__ __align__(16) uint8_t s_stage[T::kWaves][T::kStageRows(F32) * T::kPitch(F32)];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int wave = wave_all % T::kWaves, part_k = wave_all / T::kWaves;    // KS > 1: which share of K
    const int thread = wave * kWaveLanes + lane;
    const int wn = wave % WN, wm = wave / WN, g = lane >> 5;
    auto &s_buf = s_bufs[part_k];
    auto &s_scales = s_scale_sets[part_k];
    const uint32_t code_stride = static_cast<uint32_t>(kp / 2), scale_stride = static_cast<uint32_t>(kp / 32);
    // Steps of this share, and how far past its first one the row's last step
    // is: with KS > 1 the last shares may run past it, repeating it as zeros
    // (their scales are of the same row, so a NaN among them is one already).
    const int all_steps = static_cast<int>((kp + 255) / 256), steps = (all_steps + KS - 1) / KS;
    const int k_first = KS == 1 ? 0 : (part_k * steps < all_steps ? part_k * steps : all_steps - 1);
    const int k_last = all_steps - 1 - k_first, k_count = KS == 1 ? steps : all_steps - part_k * steps;
    const bool half_end = (kp & 128) != 0;       // the last step has 128 elements
    const uint32_t total = tiles_n * tiles_m;

    // The copies run two steps ahead of the products, through the tiles in
    // turn: tile pt, step pk is copied next.  A wavefront copies rows of one
    // matrix only, and thread t the scales of buffer row t: uniform bases, and
    // 32-bit offsets of the lane, row x stride (24 bits each, kp being below
    // 2^25).  Rows are clamped to the matrix: a row past the end repeats the
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
        if constexpr (KS > 1) copy_base += static_cast<uint32_t>(k_first) * 128u;
        const int r = thread - (scale_b ? 0 : BN);
        scale_src = __umul24(r < scale_last ? r : scale_last, scale_stride);
    };
    const uint32_t lds_to = lds_offset(s_buf) + wave * (T::kCopies * 1024);
    // Copy i of step pk into a buffer.  In a half step the second half of a
    // row, not used then, repeats the first.
    auto copy = [&](int i, int buf) {
        const bool half = half_end && (KS == 1 ? pk == steps - 1 : pk >= k_last);
        const uint32_t back = half ? ((chunk ^ ((i & 1) * 64u)) & 64u) : 0u;
        load_to_lds(copy_base, src[i] - back, lds_to + buf * T::kBytes + i * 1024);
    };
    const uint32_t gather = g ? 0x07050301u : 0x06040200u;
    auto scale_bytes = [&](int set, int k, int row) {
        return *(reinterpret_cast<const u32x2 *>(&s_scales[set][row]) + (k & 1));
    };

    // this lane's chunk of the first quarter step; of quarter q: ^ 32 q
    const uint32_t off = (lane & 31) * 128 + ((g ^ ((lane >> 1) & 7)) << 4);
    struct Operands {
        u32x4 n[kTN], m[kTM];
    };
    // Operand i of a quarter, in the order the products need them.
    constexpr int kReads = kTN + kTM;
    auto fetch = [&](int buf, int q, Operands &v, int i) {
        const uint32_t at = off ^ (32 * q);
        if (i == 0 || i > kTM) {
            const int r = i == 0 ? 0 : i - kTM;
            v.n[r] = *reinterpret_cast<const u32x4 *>(&s_buf[buf][(wn * kTN + r) * 4096 + at]);
        } else {
            v.m[i - 1] = *reinterpret_cast<const u32x4 *>(&s_buf[buf][BN * 128 + (wm * kTM + i - 1) * 4096 + at]);
        }
    };

    f32x16 acc[kTN][kTM];
    uint32_t sn[kTN], sm[kTM];
    // Products [FROM, TO) of a quarter, each after before(x).  Reads of LDS and
    // copies go there, one or two at a time: a wavefront issues in order, and
    // six reads in a row, from all wavefronts at once, would keep its products
    // waiting for LDS.  Each product is pinned in its place: the compiler would
    // sink products past the barrier and the branches after it, and hold all
    // four quarters' operands.
    constexpr int kBlocks = kTN * kTM, kSplit = kBlocks / 4, kRest = kBlocks - kSplit;
    auto multiply = [&](Operands &v, auto quarter, int from, int to, uint32_t mask, auto &&before) {
        constexpr int q = decltype(quarter)::value;
#pragma unroll
        for (int x = from; x < to; ++x) {
            const int i = x / kTM, j = x % kTM;
            before(x);
            if ((q >= 2 || KS > 1) && j == 0) v.n[i] &= mask;
            acc[i][j] = mfma32<q>(v.n[i], v.m[j], acc[i][j], sn[i], sm[j]);
            asm volatile("" : "+v"(acc[i][j]));
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Item c of `items` shared out over `blocks`, as early as they go evenly.
    auto share = [](int items, int blocks, int x, auto &&item) {
        const int per = (items + blocks - 1) / blocks;
#pragma unroll
        for (int c = x * per; c < (x + 1) * per && c < items; ++c) item(c);
    };
    constexpr std::integral_constant<int, 0> q0{};
    constexpr std::integral_constant<int, 1> q1{};
    constexpr std::integral_constant<int, 2> q2{};
    constexpr std::integral_constant<int, 3> q3{};

    // After the copies of step pk: with the first of two steps, the scales of
    // both go to a register (16 bytes, from a window that ends with the row, so
    // nothing past it is read), and before the next barrier settle() moves them
    // to LDS, each to its place.  Rows of less than 16 bytes, products over less
    // than 512 elements, go there at once.  Past the last tile its last copies
    // are repeated, unused.
    u32x4 next_scales{0u, 0u, 0u, 0u};
    uint32_t shift = 0;
    bool pending = false;
    int pset = 1, set = 0;       // sets of scales: the last one filled, the one in use
    auto advance = [&] {
        if (!(pk & 1)) {
            pset ^= 1;
            const uint8_t *row = scale_base + scale_src;
            if (scale_stride >= 16u) {
                const uint32_t at = static_cast<uint32_t>(k_first + pk) * 8u, end = scale_stride - 16u;
                const uint32_t from = at < end ? at : end;
                if (T::kRows == T::kTileThreads || thread < T::kRows)
                    next_scales = *reinterpret_cast<const u32x4_packed *>(row + from);
                shift = (at - from) / 4u;
                pending = true;
            } else if (thread < T::kRows) {
                for (uint32_t w = 0; w < 16; w += 4)
                    reinterpret_cast<uint32_t *>(&s_scales[pset][thread])[w / 4] =
                        w < scale_stride ? *reinterpret_cast<const uint32_t *>(row + w) : 0u;
            }
        }
        if (KS == 1 || pk < k_last) copy_base += 128;
        if (++pk == steps) {
            if (KS > 1) {                        // one tile, and every share ends together
                --pk;
                if (pk < k_last) copy_base -= 128;
            } else if (pt + gridDim.x < total) {
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
        u32x4 v = next_scales;
        if (shift & 1) v = u32x4{v.y, v.z, v.w, v.w};
        if (shift & 2) v = u32x4{v.z, v.w, v.w, v.w};
        if (thread < T::kRows) s_scales[pset][thread] = v;
        pending = false;
    };

    uint32_t t = blockIdx.x;
    if (t >= total) return;
    aim();
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) copy(i, 0);
    advance();
    settle();
    __builtin_amdgcn_s_waitcnt(0);       // this wavefront's copies have reached LDS
    __syncthreads();                     // everyone's have
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) copy(i, 1);
    advance();
    Operands v[2];
#pragma unroll
    for (int i = 0; i < kReads; ++i) fetch(0, 0, v[0], i);
    u32x2 next_n[kTN], next_m[kTM];      // scales of the step to come
    auto fetch_scales = [&](int k) {
#pragma unroll
        for (int i = 0; i < kTN; ++i) next_n[i] = scale_bytes(set, k, (wn * kTN + i) * 32 + (lane & 31));
#pragma unroll
        for (int i = 0; i < kTM; ++i) next_m[i] = scale_bytes(set, k, BN + (wm * kTM + i) * 32 + (lane & 31));
    };
    fetch_scales(0);
    int buf = 0;
    for (; t < total; t += gridDim.x) {
#pragma unroll
        for (int i = 0; i < kTN; ++i)
#pragma unroll
            for (int j = 0; j < kTM; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        // Each step starts with its first quarter and scales in registers.
        // Early in its last quarter its buffer has been read by everyone and
        // the next one has landed: the only barrier, after which the copy two
        // steps on starts and the next step's first quarter is fetched, under
        // the remaining products.
        for (int k = 0; k < steps; ++k, buf ^= 1) {
#pragma unroll
            for (int i = 0; i < kTN; ++i) sn[i] = __builtin_amdgcn_perm(next_n[i].y, next_n[i].x, gather);
#pragma unroll
            for (int i = 0; i < kTM; ++i) sm[i] = __builtin_amdgcn_perm(next_m[i].y, next_m[i].x, gather);
            const bool last = k == steps - 1;
            // a half step's second half counts as zeros (a branch around its
            // products would double the accumulators)
            const uint32_t whole = KS == 1 || k < k_count ? 0xFFFFFFFFu : 0u;
            const uint32_t second = half_end && (KS == 1 ? last : k == k_count - 1) ? 0u : whole;
            multiply(v[0], q0, 0, kBlocks, whole, [&](int x) {
                share(kReads, kBlocks, x, [&](int c) { fetch(buf, 1, v[1], c); });
            });
            multiply(v[1], q1, 0, kBlocks, whole, [&](int x) {
                share(kReads, kBlocks, x, [&](int c) { fetch(buf, 2, v[0], c); });
            });
            multiply(v[0], q2, 0, kBlocks, second, [&](int x) {
                share(kReads, kBlocks, x, [&](int c) { fetch(buf, 3, v[1], c); });
            });
            multiply(v[1], q3, 0, kSplit, second, [](int) {});
            __builtin_amdgcn_s_waitcnt(0);
            settle();
            __syncthreads();
            if ((k & 1) || last) set ^= 1;
            fetch_scales(last ? 0 : k + 1);
            multiply(v[1], q3, kSplit, kBlocks, second, [&](int x) {
                share(kReads, kRest, x - kSplit, [&](int c) { fetch(buf ^ 1, 0, v[0], c); });
                share(T::kCopies, kRest, x - kSplit, [&](int c) { copy(c, buf); });
            });
            advance();
        }

        if constexpr (KS > 1) {
            // the shares' sums, added in their order by the first one's wavefronts
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            static_assert(kTN == 1 && kTM == 1 && T::kWaves * kWaveLanes * 64 <= 2 * T::kBytes, "shares of K");
            if (part_k > 0) {
                f32x4 *to = reinterpret_cast<f32x4 *>(&s_buf[0][0]) + wave * 4 * kWaveLanes + lane;
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    to[e / 4 * kWaveLanes] = f32x4{acc[0][0][e], acc[0][0][e + 1], acc[0][0][e + 2], acc[0][0][e + 3]};
            }
            __syncthreads();
            if (part_k > 0) return;
#pragma unroll
            for (int p = 1; p < KS; ++p) {
                const f32x4 *from = reinterpret_cast<const f32x4 *>(&s_bufs[p][0][0]) + wave * 4 * kWaveLanes + lane;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f32x4 y = from[e / 4 * kWaveLanes];
                    acc[0][0][e] += y.x;
                    acc[0][0][e + 1] += y.y;
                    acc[0][0][e + 2] += y.z;
                    acc[0][0][e + 3] += y.w;
                }
            }
        }

        // Block element e of a lane is m = lane % 32, n = 8 (e / 4) +
        // 4 (lane / 32) + e % 4: 16 bytes of a row at most, where a store of
        // part of a line costs L2 as much as one of a whole line.  Each
        // wavefront turns a few rows at a time over in LDS of its own and
        // stores them in 16-byte pieces, whole lines of bf16; the next tile's
        // copies run meanwhile.
        constexpr int kEsz = F32 ? 4 : 2, kRowBytes = kTN * 32 * kEsz, kPitch = T::kPitch(F32);
        constexpr int kR = T::kStageRows(F32), kPieces = kRowBytes / 16;
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
                        // (nontemporal stores save 1-4% here and cost as
                        // much where out is read next)
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

template <bool F32, bool ROWS, bool COLS>
hipError_t quantize_layout(const MxMatrix &x, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                           uint8_t *scales_t, hipStream_t st)
{
    const int64_t row_bytes = x.row_stride * (F32 ? 4 : 2);
    const uint32_t col_tiles = static_cast<uint32_t>((mx_padded(x.cols) + kTileCols - 1) / kTileCols);
    const uint32_t row_tiles = static_cast<uint32_t>((x.rows + quant_rows(COLS) - 1) / quant_rows(COLS));
    const dim3 grid(col_tiles * row_tiles);
    const uint8_t *p = static_cast<const uint8_t *>(x.data);
    hipLaunchKernelGGL((mx_quantize_kernel<F32, ROWS, COLS>), grid, dim3(kThreads), 0, st, p, x.rows, x.cols,
                       row_bytes, row_tiles, codes, scales, codes_t, scales_t);
    return hipGetLastError();
}

template <bool F32>
hipError_t quantize_type(const MxMatrix &x, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                         uint8_t *scales_t, hipStream_t st)
{
    if (codes && codes_t) return quantize_layout<F32, true, true>(x, codes, scales, codes_t, scales_t, st);
    if (codes) return quantize_layout<F32, true, false>(x, codes, scales, codes_t, scales_t, st);
    return quantize_layout<F32, false, true>(x, codes, scales, codes_t, scales_t, st);
}

template <bool F32, int MT, int NT, typename A>
hipError_t skinny(const A &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const int64_t tiles = (b.rows + 16 * NT - 1) / (16 * NT);
    const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
    hipLaunchKernelGGL((mx_skinny_kernel<F32, MT, NT, A>), dim3(grid, static_cast<unsigned>((a.rows + 16 * MT - 1) / (16 * MT))),
                       dim3(kSkinnyWaves * kWaveLanes), 0, st, a, b, kp, out, row_bytes);
    return hipGetLastError();
}

template <bool F32, int BN, int BM, int WN, int WM, int KS = 1>
hipError_t tiles(const MxIn &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const uint32_t tn = static_cast<uint32_t>((b.rows + BN - 1) / BN);
    const uint32_t tm = static_cast<uint32_t>((a.rows + BM - 1) / BM);
    const uint64_t total = static_cast<uint64_t>(tn) * tm;
    if (total > UINT32_MAX / 2) return hipErrorInvalidValue;
    // as many workgroups as run at once (their LDS decides), each taking tiles
    // in turn; a multiple of the 8 XCDs
    constexpr unsigned kAtOnce = kCus * static_cast<unsigned>(160 * 1024 / Tile<BN, BM, WN, WM>::kLds(F32));
    if (KS > 1 && total > kCus) return hipErrorInvalidValue;     // one tile to a workgroup
    const unsigned grid = total < kAtOnce ? static_cast<unsigned>(total) : kAtOnce;
    hipLaunchKernelGGL((mx_tile_kernel<F32, BN, BM, WN, WM, KS>), dim3(grid),
                       dim3(KS * WN * WM * kWaveLanes), 0, st, a, b, kp, tn, tm, out, row_bytes);
    return hipGetLastError();
}

// Rows of B up to which a skinny product gives a workgroup 16 of them: fewer
// workgroups than that would leave CUs idle.  Above it they read A often
// enough to share it among 32 or, with more than four rows of A or rows to
// quantize on the way, 64.  (M x N x K in us, 16 / 32 / 64 rows of B: 1 x 4096 x 4096 4.4 / 6.2 / 8.9; 1 x
// 14336 x 4096 10.0 / 9.5 / 9.3; 16 x 14336 x 4096 14.0 / 11.5 / 10.4.)
constexpr int64_t kNarrow = 8192;

// Elements of K from which small tiles, one or less to a CU, split it in four
// within the workgroup.  M x N x K in us, split / not: 256 x 4096 x 14336 23.5 /
// 34.6, 512 x 1000 x 14000 20.1 / 29.4, 256 x 2048 x 5632 10.6 / 11.0, 256 x 4096
// x 4096 9.6 / 9.7, 256 x 4096 x 2048 7.8 / 6.6.
constexpr int64_t kSplitInner = 6144;

template <bool F32>
hipError_t product_type(const MxIn &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes,
                        hipStream_t st)
{
    if (a.rows <= 32 && b.rows <= kNarrow)
        return a.rows <= 16 ? skinny<F32, 1, 1>(a, b, kp, out, row_bytes, st)
                            : skinny<F32, 2, 1>(a, b, kp, out, row_bytes, st);
    if (a.rows <= 4) return skinny<F32, 1, 2>(a, b, kp, out, row_bytes, st);
    if (a.rows <= 16) return skinny<F32, 1, 4>(a, b, kp, out, row_bytes, st);
    // (17 to 32 rows over more than 8192 of B take the tiles.  The tiles / 64
    // rows of B to a skinny workgroup, from cache and, with weights in turn that
    // no cache holds, from memory: 32 x 14336 x 4096 10.9 / 11.3 and 16.0 / 12.8,
    // 32 x 28672 x 8192 27.7 / 36.7 and 39.2 / 40.0, 32 x 32000 x 2048 9.7 / 13.0
    // and 13.2 / 14.7, 17 x 9000 x 2048 5.4 / 6.1 and 9.1 / 7.2.)
    //
    // More rows, but so few tiles that each workgroup may have a CU: these split
    // K among wavefronts, which the tiles below run along (M x N x K in us, here
    // / there: 33 x 1000 x 14000 12.7 / 21.9, 64 x 2048 x 5632 7.5 / 10.7, 64 x
    // 4096 x 14336 22 / 32, 256 x 1000 x 14000 17.1 / 22.5, 128 x 1000 x 1000 4.2
    // / 5.1; with two workgroups to a CU 100 x 2048 x 5632 12.1 / 10.9).
    const int64_t m32 = (a.rows + 31) / 32;
    if (m32 * ((b.rows + 15) / 16) <= kCus) return skinny<F32, 2, 1>(a, b, kp, out, row_bytes, st);
    if (m32 * ((b.rows + 31) / 32) <= kCus) return skinny<F32, 2, 2>(a, b, kp, out, row_bytes, st);
    // The largest tile of which there are enough for the 256 CUs: a larger one
    // reads A and B less often, a smaller one leaves fewer CUs idle.  M x N x
    // K in us, tiles of 256 / 128: 5632 x 2048 x 8192 (176 tiles) 60.6 / 69.2;
    // 3000^3 (144) 28.9 / 29.5; 2048 x 4096 x 4096 (128) 32.2 / 27.7.  Of 128 /
    // 64: 1024 x 4096 x 4096 (256 tiles) 17.7 / 22.1; 1500 x 1500 x 4096 (144)
    // 18.1 / 19.4; 1024 x 1024 x 4096 (64) 13.5 / 9.5.
    const int64_t big = ((a.rows + 255) / 256) * ((b.rows + 255) / 256);
    const int64_t mid = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    if (big >= 160) return tiles<F32, 256, 256, 4, 2>(a, b, kp, out, row_bytes, st);
    if (mid >= 160) return tiles<F32, 128, 128, 2, 2>(a, b, kp, out, row_bytes, st);
    // a CU to each small tile leaves three of its wavefronts' places free: four
    // shares of K take them
    const int64_t small = ((a.rows + 63) / 64) * ((b.rows + 63) / 64);
    if (small <= kCus && kp >= kSplitInner) return tiles<F32, 64, 64, 2, 2, 4>(a, b, kp, out, row_bytes, st);
    return tiles<F32, 64, 64, 2, 2>(a, b, kp, out, row_bytes, st);
}

// Up to four rows of bf16 the linear layer's product may quantize A itself,
// every workgroup all of it, instead of in a launch before.  That costs K for
// each workgroup that a CU runs one after another, and saves a launch, so the
// rule bounds the product of the two; workgroups of 64 rows of W, which quantize
// as much for more of it, by less than those of 16.  N x K of W, in us, in the
// product / before, one row and four: 4096 x 4096 4.8 / 6.3 and 5.4 / 6.7, 4096 x
// 8192 7.7 / 8.7 and 8.7 / 9.5, 4096 x 10240 9.0 / 8.8 and 10.0 / 9.6, 4096 x
// 14336 11.9 / 10.8 and 13.0 / 12.1; two workgroups to a CU: 8192 x 4096 7.4 / 7.8
// and 8.4 / 8.5, 8192 x 5120 8.9 / 8.8 and 10.2 / 9.6, 8192 x 8192 13.7 / 12.5 and
// 15.7 / 13.7; of 64 rows: 14336 x 4096 10.4 / 11.4 and 11.0 / 12.2, 16384 x 7168
// 16.1 / 16.3 and 16.6 / 17.2; two of them: 32000 x 2048 9.7 / 11.6 and 10.2 /
// 12.2, 18000 x 4096 15.9 / 14.5 and 17.6 / 15.6, 20480 x 5120 19.4 / 16.7 and
// 20.5 / 17.9.  (Of the sizes tried the rule is wrong just above 8192 rows with a
// long K, where workgroups of 64 leave half of the CUs idle: one row of 8200 x
// 4096 10.1 / 9.8, of 8200 x 7168 15.3 / 12.8, but of 9000 x 6144 13.5 / 14.1.)
constexpr int64_t kRawRows = 4, kRawNarrow = 8192, kRawWide = 7168;

template <bool F32>
hipError_t linear_type(const MxRaw &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes,
                       hipStream_t st)
{
    return b.rows <= kNarrow ? skinny<F32, 1, 1>(a, b, kp, out, row_bytes, st)
                             : skinny<F32, 1, 4>(a, b, kp, out, row_bytes, st);
}

}  // namespace

bool mx_linear_direct(const MxMatrix &x, int64_t n)
{
    const bool narrow = n <= kNarrow;
    const int64_t rows_at_once = kCus * (narrow ? 16 : 64), turns = (n + rows_at_once - 1) / rows_at_once;
    return !x.fp32 && x.rows <= kRawRows && x.cols > 0 && x.cols * turns <= (narrow ? kRawNarrow : kRawWide) &&
           aligned_to(x.data, 16) && x.row_stride % 8 == 0 && x.cols % 8 == 0;
}

hipError_t launch_mx_linear_direct(const MxMatrix &x, const uint8_t *w_codes, const uint8_t *w_scales,
                                   const MxMatrix &out, hipStream_t st)
{
    const MxRaw a{static_cast<const uint8_t *>(x.data), x.rows, x.row_stride * 2, x.cols};
    const MxIn b{w_codes, w_scales, out.cols};
    const int64_t kp = mx_padded(x.cols), row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    uint8_t *p = static_cast<uint8_t *>(out.data);
    return out.fp32 ? linear_type<true>(a, b, kp, p, row_bytes, st) : linear_type<false>(a, b, kp, p, row_bytes, st);
}

hipError_t launch_mx_quantize(const MxMatrix &x, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                              uint8_t *scales_t, hipStream_t st)
{
    return x.fp32 ? quantize_type<true>(x, codes, scales, codes_t, scales_t, st)
                  : quantize_type<false>(x, codes, scales, codes_t, scales_t, st);
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, const MxMatrix &out,
                                hipStream_t st)
{
    const int64_t threads = out.rows * ((out.cols + 7) / 8);
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
    uint8_t *p = static_cast<uint8_t *>(out.data);
    const int64_t row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    if (out.fp32)
        hipLaunchKernelGGL(mx_dequantize_kernel<true>, grid, dim3(kThreads), 0, st, codes, scales, out.rows,
                           out.cols, p, row_bytes);
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<false>, grid, dim3(kThreads), 0, st, codes, scales, out.rows,
                           out.cols, p, row_bytes);
    return hipGetLastError();
}

hipError_t launch_mx_product(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                             const uint8_t *b_scales, int64_t inner, const MxMatrix &out, hipStream_t st)
{
    const MxIn a{a_codes, a_scales, out.rows}, b{b_codes, b_scales, out.cols};
    const int64_t kp = mx_padded(inner), row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    uint8_t *p = static_cast<uint8_t *>(out.data);
    if (inner == 0) {
        const int64_t blocks = (out.rows * out.cols + kThreads - 1) / kThreads;
        const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
        if (out.fp32) hipLaunchKernelGGL(zero_kernel<true>, grid, dim3(kThreads), 0, st, out.rows, out.cols, p, row_bytes);
        else hipLaunchKernelGGL(zero_kernel<false>, grid, dim3(kThreads), 0, st, out.rows, out.cols, p, row_bytes);
        return hipGetLastError();
    }
    return out.fp32 ? product_type<true>(a, b, kp, p, row_bytes, st)
                    : product_type<false>(a, b, kp, p, row_bytes, st);
}

}  // namespace flashopt
