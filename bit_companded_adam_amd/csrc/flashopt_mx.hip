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
#include "flashopt_internal.h"

namespace flashopt {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = kBlockThreads;

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// fp32 -> bf16, round to nearest even (no NaN keeps its payload's low half:
// the quiet bit is set).
__device__ __forceinline__ uint32_t bf16_rne(float x)
{
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// -------------------------------------------------------------- quantize

// The scale byte of a group from its largest biased exponent E (255: the
// group holds an infinity or NaN, and so does its scale), and 2^(127 - byte),
// the exact reciprocal of the scale (0 for byte 255).
__device__ __forceinline__ uint32_t scale_byte(uint32_t e)
{
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
__device__ __forceinline__ float scale_recip(uint32_t byte)
{
    return __uint_as_float((byte == 255u ? 0u : 254u - byte) << 23);
}

// Two E2M1 codes in byte SEL of acc (v_cvt_scalef32_pk_fp4_f32: half to even,
// saturating at 6).
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t acc, float a, float b)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(acc, a, b, 1.0f, SEL);
}

__device__ __forceinline__ uint32_t codes8(const float (&y)[8])
{
    uint32_t w = codes2<0>(0u, y[0], y[1]);
    w = codes2<1>(w, y[2], y[3]);
    w = codes2<2>(w, y[4], y[5]);
    return codes2<3>(w, y[6], y[7]);
}

// A wavefront takes 32 rows by 256 columns, four columns to a lane: every
// load covers 512 (bf16) or 1024 bytes of a row, a group along a row is
// eight lanes, and a group along a column is one lane's 32 values.
constexpr int kLaneCols = 4;
constexpr int kTileCols = 64 * kLaneCols;
constexpr int kWaveRows = 32;
constexpr int kTileRows = kWaveRows * (kThreads / kWaveLanes);

// Four elements of a row as fp32 bit patterns; columns past the end are 0.
template <bool F32, bool VEC>
__device__ __forceinline__ void load4(const uint8_t *row, int64_t c, int64_t cols, uint32_t (&w)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = 0u;
    if constexpr (VEC) {
        if (c + 4 <= cols) {
            if constexpr (F32) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(row + c * 4);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(row + c * 2);
                w[0] = v.x << 16; w[1] = v.x & 0xFFFF0000u;
                w[2] = v.y << 16; w[3] = v.y & 0xFFFF0000u;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (c + j >= cols) continue;
        if constexpr (F32) w[j] = reinterpret_cast<const uint32_t *>(row)[c + j];
        else w[j] = static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[c + j]) << 16;
    }
}

__device__ __forceinline__ uint32_t exponent(uint32_t bits) { return (bits >> 23) & 0xFFu; }

// Maximum over aligned groups of eight lanes.
__device__ __forceinline__ uint32_t max8(uint32_t x)
{
    x = umax32(x, __shfl_xor(x, 1, kWaveLanes));
    x = umax32(x, __shfl_xor(x, 2, kWaveLanes));
    return umax32(x, __shfl_xor(x, 4, kWaveLanes));
}

// Codes of x along its rows (ROWS) and of its transpose (COLS), from one read.
template <bool F32, bool ROWS, bool COLS, bool VEC>
__global__ void __launch_bounds__(kThreads)
mx_quantize_kernel(const uint8_t *__restrict__ x, int64_t rows, int64_t cols, int64_t row_bytes,
                   uint32_t col_tiles, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t)
{
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = threadIdx.x / kWaveLanes;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / col_tiles) * kTileRows + wave * kWaveRows;
    const int64_t c = static_cast<int64_t>(blockIdx.x % col_tiles) * kTileCols + lane * kLaneCols;
    const int64_t colsp = mx_padded(cols), rowsp = mx_padded(rows);

    uint32_t w[kWaveRows][kLaneCols];
#pragma unroll
    for (int r = 0; r < kWaveRows; ++r) {
        if (row0 + r < rows) {
            load4<F32, VEC>(x + (row0 + r) * row_bytes, c, cols, w[r]);
        } else {
#pragma unroll
            for (int j = 0; j < kLaneCols; ++j) w[r][j] = 0u;
        }
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int r = 0; r < kWaveRows; ++r) {
            if (row0 + r >= rows) break;
            const uint32_t e = max8(umax32(umax32(exponent(w[r][0]), exponent(w[r][1])),
                                           umax32(exponent(w[r][2]), exponent(w[r][3]))));
            const uint32_t b = scale_byte(e);
            const float f = scale_recip(b);
            uint32_t q = codes2<0>(0u, __uint_as_float(w[r][0]) * f, __uint_as_float(w[r][1]) * f);
            q = codes2<1>(q, __uint_as_float(w[r][2]) * f, __uint_as_float(w[r][3]) * f);
            if (b == 255u) q = 0u;
            if (c < colsp) {
                *reinterpret_cast<uint16_t *>(codes + (row0 + r) * (colsp / 2) + c / 2) =
                    static_cast<uint16_t>(q);
                if ((lane & 7) == 0)
                    scales[(row0 + r) * (colsp / 32) + c / 32] = static_cast<uint8_t>(b);
            }
        }
    }
    if constexpr (COLS) {
#pragma unroll
        for (int j = 0; j < kLaneCols; ++j) {
            uint32_t e = 0u;
#pragma unroll
            for (int r = 0; r < kWaveRows; ++r) e = umax32(e, exponent(w[r][j]));
            const uint32_t b = scale_byte(e);
            const float f = scale_recip(b);
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(w[8 * k + i][j]) * f;
                q[k] = b == 255u ? 0u : codes8(y);
            }
            if (c + j < cols) {
                *reinterpret_cast<u32x4 *>(codes_t + (c + j) * (rowsp / 2) + row0 / 2) =
                    u32x4{q[0], q[1], q[2], q[3]};
                scales_t[(c + j) * (rowsp / 32) + row0 / 32] = static_cast<uint8_t>(b);
            }
        }
    }
}

// ------------------------------------------------------------ dequantize

// The value of a scale byte: 2^(b - 127), subnormal at b = 0, NaN at 255.
__device__ __forceinline__ float scale_value(uint32_t b)
{
    if (b == 0u) return __uint_as_float(0x00400000u);
    return __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);
}

// One thread per eight columns.
template <bool F32, bool VEC>
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
        if (VEC && c + 8 <= cols) {
            if constexpr (F32) {
                *reinterpret_cast<f32x4 *>(o + c * 4) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4 *>(o + c * 4 + 16) = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                u32x4 p;
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = bf16_rne(v[2 * k]) | (bf16_rne(v[2 * k + 1]) << 16);
                *reinterpret_cast<u32x4 *>(o + c * 2) = p;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c + k >= cols) break;
                if constexpr (F32) reinterpret_cast<float *>(o)[c + k] = v[k];
                else reinterpret_cast<uint16_t *>(o)[c + k] = static_cast<uint16_t>(bf16_rne(v[k]));
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

// Four consecutive outputs of row m from column n on.
template <bool F32, bool VEC>
__device__ __forceinline__ void store4(uint8_t *out, int64_t row_bytes, int64_t m, int64_t n, int64_t cols,
                                       float a, float b, float c, float d)
{
    uint8_t *o = out + m * row_bytes;
    if (VEC && n + 4 <= cols) {
        if constexpr (F32) {
            *reinterpret_cast<f32x4 *>(o + n * 4) = f32x4{a, b, c, d};
        } else {
            *reinterpret_cast<u32x2 *>(o + n * 2) =
                u32x2{bf16_rne(a) | (bf16_rne(b) << 16), bf16_rne(c) | (bf16_rne(d) << 16)};
        }
        return;
    }
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= cols) break;
        if constexpr (F32) reinterpret_cast<float *>(o)[n + i] = v[i];
        else reinterpret_cast<uint16_t *>(o)[n + i] = static_cast<uint16_t>(bf16_rne(v[i]));
    }
}

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

// Few rows of A (at most 16 MT): the time is B's, read once, so nothing is
// staged.  A workgroup takes 16 NT rows of B; its wavefronts take 256-element
// steps of K in turn and add their sums at the end, in wavefront order.
// Within a step a lane holds groups 2 g and 2 g + 1 of its row (g = lane / 16):
// 32 consecutive bytes, and any assignment of groups to the instruction's
// four K slots is the same sum as long as both operands and their scales
// agree.
constexpr int kSkinnyWaves = kThreads / kWaveLanes;

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

template <bool F32, bool VEC, int MT, int NT>
__global__ void __launch_bounds__(kThreads)
mx_skinny_kernel(MxIn a, MxIn b, int64_t kp, uint8_t *__restrict__ out, int64_t row_bytes)
{
    __shared__ f32x4 s_acc[kSkinnyWaves][NT][MT][kWaveLanes];
    const int lane = threadIdx.x & (kWaveLanes - 1), wave = threadIdx.x / kWaveLanes;
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t tiles = (b.rows + 16 * NT - 1) / (16 * NT), steps = (kp + 255) / 256;
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
            arow[t] = 16 * t + l16;
            if (arow[t] >= a.rows) arow[t] = a.rows - 1;
        }
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t k = wave; k < steps; k += kSkinnyWaves) {
            Step sb[NT], sa[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) sb[i] = load_step(b, brow[i], kp, k * 8 + 2 * g);
#pragma unroll
            for (int j = 0; j < MT; ++j) sa[j] = load_step(a, arow[j], kp, k * 8 + 2 * g);
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
            const int64_t m = 16 * (i % MT) + l16, n = n0 + 16 * (i / MT) + 4 * g;
            if (m < a.rows) store4<F32, VEC>(out, row_bytes, m, n, b.rows, v.x, v.y, v.z, v.w);
        }
        __syncthreads();
    }
}

// Larger products: a workgroup computes a BN x BM tile of out^T, its
// wavefronts in a WN x WM arrangement of 32 x 32 accumulator blocks.
//
// Each K step of 256 elements is 128 bytes of every row, one cache line,
// copied from global memory to LDS by the DMA (16 bytes to a lane, eight rows
// an instruction).  LDS holds row r's 16-byte chunk c at slot c ^ (r & 7) of
// the row's 128 bytes: the DMA writes lanes in order, so each lane fetches
// the chunk that belongs to its slot, and the 32 rows that an operand read
// takes at one c then fall on all banks.  Two buffers: the copy of the next
// step runs while this one is multiplied, one barrier a step.
//
// Scales go straight to registers, eight bytes of a row and step; the four
// that a lane needs (groups 2 k + lane / 32) are gathered into one word with
// a byte permutation, from which the instruction selects by an immediate.
typedef __attribute__((address_space(1))) const uint8_t g_u8;
typedef __attribute__((address_space(3))) uint8_t l_u8;

template <int BN, int BM, int WN, int WM>
struct Tile {
    static constexpr int kWaves = WN * WM;
    static constexpr int kTileThreads = kWaves * kWaveLanes;
    static constexpr int kRows = BN + BM;                  // rows of B, then of A
    static constexpr int kBytes = kRows * 128;             // one buffer
    static constexpr int kCopies = kRows / 8 / kWaves;     // DMA instructions of a wavefront and step
    static constexpr int kTN = BN / WN / 32, kTM = BM / WM / 32;
    static_assert(kRows % (8 * kWaves) == 0 && BN % (32 * WN) == 0 && BM % (32 * WM) == 0, "tile");
};

// The tile of this workgroup: neighbours on one XCD (workgroup b runs on XCD
// b % 8) take neighbouring tiles, in columns of kGroupM tiles, so that the
// 32 or so that run together share their rows in the XCD's L2.
constexpr uint32_t kGroupM = 4;

__device__ __forceinline__ void tile_of_block(uint32_t tiles_n, uint32_t tiles_m, uint32_t &tn, uint32_t &tm)
{
    const uint32_t nb = gridDim.x, b = blockIdx.x, x = b % 8u;
    const uint32_t per = (nb + 7u) / 8u, full = nb % 8u;
    uint32_t lb = x * per + b / 8u;
    if (full != 0u && x > full) lb -= x - full;
    const uint32_t group = lb / (kGroupM * tiles_n), first = group * kGroupM;
    const uint32_t width = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
    const uint32_t in = lb - group * kGroupM * tiles_n;
    tm = first + in % width;
    tn = in / width;
}

template <bool F32, bool VEC, int BN, int BM, int WN, int WM>
__global__ void __launch_bounds__(WN *WM *kWaveLanes)
mx_tile_kernel(MxIn a, MxIn b, int64_t kp, uint32_t tiles_n, uint32_t tiles_m, uint8_t *__restrict__ out,
               int64_t row_bytes)
{
    using T = Tile<BN, BM, WN, WM>;
    __shared__ __align__(128) uint8_t s_buf[2][T::kBytes];
    const int lane = threadIdx.x & (kWaveLanes - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int wn = wave % WN, wm = wave / WN;
    uint32_t tile_n, tile_m;
    tile_of_block(tiles_n, tiles_m, tile_n, tile_m);
    const int64_t n0 = static_cast<int64_t>(tile_n) * BN, m0 = static_cast<int64_t>(tile_m) * BM;
    const uint32_t code_stride = static_cast<uint32_t>(kp / 2), scale_stride = static_cast<uint32_t>(kp / 32);

    // this lane's rows of the copies, clamped to the matrices: a row past the
    // end repeats the last one and is not stored
    const uint8_t *src[T::kCopies];
    const int slot_chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
        const int r = (wave * T::kCopies + i) * 8 + (lane >> 3);      // row of the buffer
        const bool is_b = (wave * T::kCopies + i) * 8 < BN;
        const MxIn &in = is_b ? b : a;
        int64_t row = is_b ? n0 + r : m0 + r - BN;
        if (row >= in.rows) row = in.rows - 1;
        src[i] = in.codes + row * code_stride;
    }
    const uint8_t *scale_n[T::kTN], *scale_m[T::kTM];
#pragma unroll
    for (int i = 0; i < T::kTN; ++i) {
        int64_t row = n0 + (wn * T::kTN + i) * 32 + (lane & 31);
        if (row >= b.rows) row = b.rows - 1;
        scale_n[i] = b.scales + row * scale_stride;
    }
#pragma unroll
    for (int i = 0; i < T::kTM; ++i) {
        int64_t row = m0 + (wm * T::kTM + i) * 32 + (lane & 31);
        if (row >= a.rows) row = a.rows - 1;
        scale_m[i] = a.scales + row * scale_stride;
    }
    const int g = lane >> 5;
    const uint32_t gather = g ? 0x07050301u : 0x06040200u;

    const int64_t steps = (kp + 255) / 256;
    const bool half_end = (kp & 128) != 0;       // the last step has 128 elements

    auto copy = [&](int64_t k, int buf) {
        // the second half of a half step repeats the first: it is not used
        const int chunk = (half_end && k == steps - 1) ? (slot_chunk & 3) : slot_chunk;
#pragma unroll
        for (int i = 0; i < T::kCopies; ++i) {
            const uint8_t *p = src[i] + k * 128 + chunk * 16;
            uint8_t *l = &s_buf[buf][(wave * T::kCopies + i) * 1024];
            __builtin_amdgcn_global_load_lds((g_u8 *)p, (l_u8 *)l, 16, 0, 0);
        }
    };
    auto scale_word = [&](const uint8_t *p, int64_t k) {
        const uint32_t lo = *reinterpret_cast<const uint32_t *>(p + k * 8);
        const uint32_t hi = *reinterpret_cast<const uint32_t *>(
            p + k * 8 + ((half_end && k == steps - 1) ? 0 : 4));
        return __builtin_amdgcn_perm(hi, lo, gather);
    };

    f32x16 acc[T::kTN][T::kTM];
#pragma unroll
    for (int i = 0; i < T::kTN; ++i)
#pragma unroll
        for (int j = 0; j < T::kTM; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    uint32_t off[4];             // this lane's chunk of each quarter step
#pragma unroll
    for (int q = 0; q < 4; ++q) off[q] = (lane & 31) * 128 + (((2 * q + g) ^ (lane & 7)) << 4);

    auto multiply = [&](int buf, const uint32_t (&sn)[T::kTN], const uint32_t (&sm)[T::kTM], auto quarter) {
        constexpr int q = decltype(quarter)::value;
        u32x4 vn[T::kTN], vm[T::kTM];
#pragma unroll
        for (int i = 0; i < T::kTN; ++i)
            vn[i] = *reinterpret_cast<const u32x4 *>(&s_buf[buf][(wn * T::kTN + i) * 4096 + off[q]]);
#pragma unroll
        for (int i = 0; i < T::kTM; ++i)
            vm[i] = *reinterpret_cast<const u32x4 *>(&s_buf[buf][BN * 128 + (wm * T::kTM + i) * 4096 + off[q]]);
#pragma unroll
        for (int i = 0; i < T::kTN; ++i)
#pragma unroll
            for (int j = 0; j < T::kTM; ++j) acc[i][j] = mfma32<q>(vn[i], vm[j], acc[i][j], sn[i], sm[j]);
    };

    if (steps > 0) copy(0, 0);
    for (int64_t k = 0; k < steps; ++k) {
        const int buf = static_cast<int>(k & 1);
        uint32_t sn[T::kTN], sm[T::kTM];
#pragma unroll
        for (int i = 0; i < T::kTN; ++i) sn[i] = scale_word(scale_n[i], k);
#pragma unroll
        for (int i = 0; i < T::kTM; ++i) sm[i] = scale_word(scale_m[i], k);
        __builtin_amdgcn_s_waitcnt(0);   // this wavefront's copies have reached LDS
        __syncthreads();                 // everyone's have, and the other buffer is free
        if (k + 1 < steps) copy(k + 1, buf ^ 1);
        multiply(buf, sn, sm, std::integral_constant<int, 0>{});
        multiply(buf, sn, sm, std::integral_constant<int, 1>{});
        if (!(half_end && k == steps - 1)) {
            multiply(buf, sn, sm, std::integral_constant<int, 2>{});
            multiply(buf, sn, sm, std::integral_constant<int, 3>{});
        }
    }

    // block element e of a lane: m = lane % 32, n = 8 (e / 4) + 4 (lane / 32) + e % 4
#pragma unroll
    for (int j = 0; j < T::kTM; ++j) {
        const int64_t m = m0 + (wm * T::kTM + j) * 32 + (lane & 31);
        if (m >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < T::kTN; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                store4<F32, VEC>(out, row_bytes, m, n0 + (wn * T::kTN + i) * 32 + 2 * e + 4 * g, b.rows,
                                 acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
    }
}

// ------------------------------------------------------------- launching

bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool F32, bool ROWS, bool COLS>
hipError_t quantize_layout(const MxMatrix &x, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                           uint8_t *scales_t, hipStream_t st)
{
    const int64_t row_bytes = x.row_stride * (F32 ? 4 : 2);
    const uint32_t col_tiles = static_cast<uint32_t>((mx_padded(x.cols) + kTileCols - 1) / kTileCols);
    const uint32_t row_tiles = static_cast<uint32_t>((x.rows + kTileRows - 1) / kTileRows);
    const dim3 grid(col_tiles * row_tiles);
    const uint8_t *p = static_cast<const uint8_t *>(x.data);
    constexpr int vec = F32 ? 16 : 8;
    if (aligned_to(p, vec) && row_bytes % vec == 0)
        hipLaunchKernelGGL((mx_quantize_kernel<F32, ROWS, COLS, true>), grid, dim3(kThreads), 0, st, p, x.rows,
                           x.cols, row_bytes, col_tiles, codes, scales, codes_t, scales_t);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<F32, ROWS, COLS, false>), grid, dim3(kThreads), 0, st, p, x.rows,
                           x.cols, row_bytes, col_tiles, codes, scales, codes_t, scales_t);
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

template <bool F32, bool VEC, int MT, int NT>
hipError_t skinny(const MxIn &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const int64_t tiles = (b.rows + 16 * NT - 1) / (16 * NT);
    const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
    hipLaunchKernelGGL((mx_skinny_kernel<F32, VEC, MT, NT>), dim3(grid), dim3(kThreads), 0, st, a, b, kp, out,
                       row_bytes);
    return hipGetLastError();
}

template <bool F32, bool VEC, int BN, int BM, int WN, int WM>
hipError_t tiles(const MxIn &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes, hipStream_t st)
{
    const uint32_t tn = static_cast<uint32_t>((b.rows + BN - 1) / BN);
    const uint32_t tm = static_cast<uint32_t>((a.rows + BM - 1) / BM);
    const uint64_t grid = static_cast<uint64_t>(tn) * tm;
    if (grid * (WN * WM * kWaveLanes) > UINT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((mx_tile_kernel<F32, VEC, BN, BM, WN, WM>), dim3(static_cast<unsigned>(grid)),
                       dim3(WN * WM * kWaveLanes), 0, st, a, b, kp, tn, tm, out, row_bytes);
    return hipGetLastError();
}

template <bool F32, bool VEC>
hipError_t product_type(const MxIn &a, const MxIn &b, int64_t kp, uint8_t *out, int64_t row_bytes,
                        hipStream_t st)
{
    if (a.rows <= 16) return skinny<F32, VEC, 1, 2>(a, b, kp, out, row_bytes, st);
    if (a.rows <= 32) return skinny<F32, VEC, 2, 2>(a, b, kp, out, row_bytes, st);
    const int64_t big = ((a.rows + 255) / 256) * ((b.rows + 255) / 256);
    const int64_t mid = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    if (big >= 200) return tiles<F32, VEC, 256, 256, 4, 2>(a, b, kp, out, row_bytes, st);
    if (mid >= 200) return tiles<F32, VEC, 128, 128, 2, 2>(a, b, kp, out, row_bytes, st);
    return tiles<F32, VEC, 64, 64, 2, 2>(a, b, kp, out, row_bytes, st);
}

}  // namespace

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
    const bool vec = aligned_to(p, 16) && row_bytes % 16 == 0;
    if (out.fp32 && vec)
        hipLaunchKernelGGL((mx_dequantize_kernel<true, true>), grid, dim3(kThreads), 0, st, codes, scales,
                           out.rows, out.cols, p, row_bytes);
    else if (out.fp32)
        hipLaunchKernelGGL((mx_dequantize_kernel<true, false>), grid, dim3(kThreads), 0, st, codes, scales,
                           out.rows, out.cols, p, row_bytes);
    else if (vec)
        hipLaunchKernelGGL((mx_dequantize_kernel<false, true>), grid, dim3(kThreads), 0, st, codes, scales,
                           out.rows, out.cols, p, row_bytes);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<false, false>), grid, dim3(kThreads), 0, st, codes, scales,
                           out.rows, out.cols, p, row_bytes);
    return hipGetLastError();
}

hipError_t launch_mx_product(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                             const uint8_t *b_scales, int64_t inner, const MxMatrix &out, hipStream_t st)
{
    const MxIn a{a_codes, a_scales, out.rows}, b{b_codes, b_scales, out.cols};
    const int64_t kp = mx_padded(inner), row_bytes = out.row_stride * (out.fp32 ? 4 : 2);
    uint8_t *p = static_cast<uint8_t *>(out.data);
    const int need = out.fp32 ? 16 : 8;
    const bool vec = aligned_to(p, need) && row_bytes % need == 0;
    if (out.fp32) return vec ? product_type<true, true>(a, b, kp, p, row_bytes, st)
                             : product_type<true, false>(a, b, kp, p, row_bytes, st);
    return vec ? product_type<false, true>(a, b, kp, p, row_bytes, st)
               : product_type<false, false>(a, b, kp, p, row_bytes, st);
}

}  // namespace flashopt
