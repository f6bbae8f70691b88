// Device code that the kernels of quantized matrices share (flashopt_mx.hip,
// flashopt_fp8.hip, flashopt_norm.hip): vector types, bf16 roundings, the order
// of tiles over the XCDs, stores of a product's outputs, copies to LDS.
#ifndef FLASHOPT_DEVICE_H
#define FLASHOPT_DEVICE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flashopt_internal.h"

namespace flashopt {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
// Vectors at any address that their elements may have: global loads and stores
// of these widths need no alignment.  (8191 x 5631 x 2048 takes 68 us with
// such stores of out, 125 with one an element; 8192 x 5632 64.)
typedef u32x4 u32x4_packed __attribute__((aligned(2)));
typedef u32x2 u32x2_packed __attribute__((aligned(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = kBlockThreads;
constexpr unsigned kCus = 256;

// Number b of nb workgroups renumbered so that each of the 8 XCDs (workgroup b
// runs on XCD b % 8) takes one contiguous eighth of them.
__device__ __forceinline__ uint32_t xcd_contiguous(uint32_t b, uint32_t nb)
{
    const uint32_t x = b % 8u, per = (nb + 7u) / 8u, full = nb % 8u;
    return x * per + b / 8u - (full != 0u && x > full ? x - full : 0u);
}

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// fp32 -> bf16, round to nearest even (v_cvt_pk_bf16_f32): one value, or two
// to a word.
__device__ __forceinline__ uint16_t bf16_rne(float x)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// Four consecutive outputs of row m from column n on.
template <bool F32>
__device__ __forceinline__ void store4(uint8_t *out, int64_t row_bytes, int64_t m, int64_t n, int64_t cols,
                                       float a, float b, float c, float d)
{
    uint8_t *o = out + m * row_bytes;
    if (n + 4 <= cols) {
        if constexpr (F32) {
            *reinterpret_cast<u32x4_packed *>(o + n * 4) =
                u32x4{__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
        } else {
            *reinterpret_cast<u32x2_packed *>(o + n * 2) = u32x2{bf16_pair(a, b), bf16_pair(c, d)};
        }
        return;
    }
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= cols) break;
        if constexpr (F32) reinterpret_cast<float *>(o)[n + i] = v[i];
        else reinterpret_cast<uint16_t *>(o)[n + i] = bf16_rne(v[i]);
    }
}

typedef __attribute__((address_space(3))) uint8_t l_u8;

// 16 bytes a lane from base + offset to LDS, the lanes' in order from byte
// `to` on.  Written out because the compiler, which cannot tell the buffers
// apart, would wait for the copy before any read of LDS; it has no register
// result, and the kernel waits for it (vmcnt 0) ahead of the barrier that
// publishes it.  M0 holds the LDS address; nothing else in a kernel that calls
// this uses it (it is a reserved register, which an asm cannot name as
// clobbered).
__device__ __forceinline__ uint32_t lds_offset(const void *p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((l_u8 *)p));
}
__device__ __forceinline__ void load_to_lds(const uint8_t *base, uint32_t offset, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(offset), "s"(base)
                 : "memory");
}

// Tile number t of a launch: neighbours on one XCD take neighbouring tiles,
// in columns of kGroupM tiles, so that the 32 or so that run together share
// their rows in the XCD's L2 (columns of 8 are level).
constexpr uint32_t kGroupM = 4;

__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_n, uint32_t tiles_m, uint32_t &tn, uint32_t &tm)
{
    const uint32_t lb = xcd_contiguous(t, tiles_n * tiles_m);
    const uint32_t group = lb / (kGroupM * tiles_n), first = group * kGroupM;
    const uint32_t width = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
    const uint32_t in = lb - group * kGroupM * tiles_n;
    tm = first + in % width;
    tn = in / width;
}

// out = 0, for a product over nothing.
template <bool F32>
__global__ void __launch_bounds__(kThreads)
zero_kernel(int64_t rows, int64_t cols, uint8_t *__restrict__ out, int64_t row_bytes)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < rows * cols;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        uint8_t *o = out + i / cols * row_bytes;
        if constexpr (F32) reinterpret_cast<float *>(o)[i % cols] = 0.0f;
        else reinterpret_cast<uint16_t *>(o)[i % cols] = 0;
    }
}

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace flashopt

#endif  // FLASHOPT_DEVICE_H
