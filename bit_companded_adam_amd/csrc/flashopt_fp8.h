// Device code of the 8-bit matrices (flashopt_fp8.hip, flashopt_norm.hip): a
// group's scale, its codes, and the eight consecutive values of a row that a
// lane holds.
//
// A group is 128 elements along a row (or a block of 128 x 128): sixteen
// lanes, one row of a wavefront's DPP operations.  With E the biased exponent
// of its largest magnitude and f that one's fraction in [1, 2), the scale is
// 2^(E - 127 - T), T the exponent of the format's largest value 1.75 x 2^T (448
// or 57344), one more for f > 1.75: no value saturates.  The stored byte is not
// below 0, 2^-127.
#ifndef FLASHOPT_FP8_H
#define FLASHOPT_FP8_H

#include <type_traits>

#include "flashopt_device.h"

namespace flashopt {
namespace {

typedef int16_t s16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kInfinite = 0x7F800000u;      // magnitudes from here on are infinities and NaN
constexpr uint32_t kNanByte = 255u;

// The scale as an fp32 pattern (field 0 is 2^-127 to the conversions, which
// read the exponent field alone) of a group with largest magnitude pattern
// `top`; the carry out of the fraction is f > 1.75.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_scale(uint32_t top)
{
    constexpr uint32_t kTop = FMT == kE5M2 ? 15u : 8u;
    return __builtin_elementwise_sub_sat((top + 0x1FFFFFu) & kInfinite, kTop << 23);
}

// Two codes, half to even, in one half of acc: from fp32 values, or from a
// word of two bf16 ones.
template <int FMT, bool HIGH>
__device__ __forceinline__ uint32_t fp8_codes(uint32_t acc, uint32_t a, uint32_t b, uint32_t scale)
{
    const s16x2 o = __builtin_bit_cast(s16x2, acc);
    const float x = __uint_as_float(a), y = __uint_as_float(b), s = __uint_as_float(scale);
    if constexpr (FMT == kE5M2)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(o, x, y, s, HIGH));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, x, y, s, HIGH));
}
template <int FMT, bool HIGH>
__device__ __forceinline__ uint32_t fp8_codes(uint32_t acc, uint32_t ab, uint32_t scale)
{
    const s16x2 o = __builtin_bit_cast(s16x2, acc);
    const bf16x2 x = __builtin_bit_cast(bf16x2, ab);
    const float s = __uint_as_float(scale);
    if constexpr (FMT == kE5M2)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(o, x, s, HIGH));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, x, s, HIGH));
}

// Eight consecutive values of a row, in the words they came in.
template <bool F32>
struct Eight {
    uint32_t w[F32 ? 8 : 4];
};

template <bool F32, bool STREAM>
__device__ __forceinline__ Eight<F32> load8(const uint8_t *p)
{
    Eight<F32> f;
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
        const u32x4_packed *at = reinterpret_cast<const u32x4_packed *>(p + 16 * i);
        const u32x4 v = STREAM ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
        for (int k = 0; k < 4; ++k) f.w[4 * i + k] = v[k];
    }
    return f;
}
template <bool F32>
__device__ __forceinline__ void load1(Eight<F32> &f, int j, const uint8_t *p)
{
    if constexpr (F32) f.w[j] = *reinterpret_cast<const uint32_t *>(p + j * 4);
    else f.w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p + j * 2)) << (16 * (j & 1));
}
// The first `count` of the eight, zeros for the others.
template <bool F32, bool STREAM>
__device__ __forceinline__ Eight<F32> load8(const uint8_t *p, int64_t count)
{
    if (count >= 8) return load8<F32, STREAM>(p);
    Eight<F32> f{};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < count) load1<F32>(f, j, p);
    return f;
}
template <bool F32>
__device__ __forceinline__ void store8(uint8_t *p, const Eight<F32> &f, int64_t count)
{
    if (count >= 8) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            *reinterpret_cast<u32x4_packed *>(p + 16 * i) =
                u32x4{f.w[4 * i], f.w[4 * i + 1], f.w[4 * i + 2], f.w[4 * i + 3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= count) break;
        if constexpr (F32) reinterpret_cast<uint32_t *>(p)[j] = f.w[j];
        else reinterpret_cast<uint16_t *>(p)[j] = static_cast<uint16_t>(f.w[j / 2] >> (16 * (j & 1)));
    }
}

template <bool F32>
__device__ __forceinline__ float value(const Eight<F32> &f, int j)
{
    if constexpr (F32) return __uint_as_float(f.w[j]);
    return __uint_as_float((j & 1) ? f.w[j / 2] & 0xFFFF0000u : f.w[j / 2] << 16);
}
// fp32 values rounded to a row's type (bf16: to nearest even).
template <bool F32>
__device__ __forceinline__ Eight<F32> rounded8(const float (&v)[8])
{
    Eight<F32> f;
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i)
        f.w[i] = F32 ? __float_as_uint(v[i]) : bf16_pair(v[2 * i], v[2 * i + 1]);
    return f;
}

// Magnitude patterns, word by word; bf16 ones stay two to a word.
template <bool F32>
__device__ __forceinline__ void raise(Eight<F32> &a, const Eight<F32> &b)
{
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i)
        a.w[i] = F32 ? umax32(a.w[i], b.w[i] & 0x7FFFFFFFu) : max_u16(a.w[i], b.w[i] & 0x7FFF7FFFu);
}
// The largest of eight magnitudes, as an fp32 pattern.
template <bool F32>
__device__ __forceinline__ uint32_t largest(const Eight<F32> &m)
{
    if constexpr (F32)
        return umax32(umax32(umax32(m.w[0], m.w[1]), umax32(m.w[2], m.w[3])),
                      umax32(umax32(m.w[4], m.w[5]), umax32(m.w[6], m.w[7])));
    const uint32_t t = max_u16(max_u16(m.w[0], m.w[1]), max_u16(m.w[2], m.w[3]));
    return umax32(t & 0xFFFF0000u, t << 16);
}
template <bool F32>
__device__ __forceinline__ uint32_t largest_of(const Eight<F32> &f)
{
    Eight<F32> m{};
    raise(m, f);
    return largest(m);
}

// A lane's eight codes.
template <bool F32, int FMT>
__device__ __forceinline__ u32x2 row_codes(const Eight<F32> &f, uint32_t scale)
{
    u32x2 q;
    if constexpr (F32) {
        q.x = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f.w[0], f.w[1], scale), f.w[2], f.w[3], scale);
        q.y = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f.w[4], f.w[5], scale), f.w[6], f.w[7], scale);
    } else {
        q.x = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f.w[0], scale), f.w[1], scale);
        q.y = fp8_codes<FMT, true>(fp8_codes<FMT, false>(0u, f.w[2], scale), f.w[3], scale);
    }
    return q;
}

// Maximum over the sixteen lanes that hold a group.
template <int ROR>
__device__ __forceinline__ uint32_t rotated(uint32_t x)
{
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x120 + ROR, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t max16(uint32_t x)
{
    x = umax32(x, rotated<1>(x));
    x = umax32(x, rotated<2>(x));
    x = umax32(x, rotated<4>(x));
    return umax32(x, rotated<8>(x));
}
// What lanes l, l ^ 16, l ^ 32 and l ^ 48 hold, combined.
template <typename F>
__device__ __forceinline__ uint32_t across16(uint32_t x, F &&combine)
{
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = combine(static_cast<uint32_t>(a[0]), static_cast<uint32_t>(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return combine(static_cast<uint32_t>(b[0]), static_cast<uint32_t>(b[1]));
}

// Sum over a wavefront, known to all of its lanes.
__device__ __forceinline__ float wave_sum(float x)
{
    auto turned = [](float v, auto by) {
        return __uint_as_float(rotated<decltype(by)::value>(__float_as_uint(v)));
    };
    x += turned(x, std::integral_constant<int, 1>{});
    x += turned(x, std::integral_constant<int, 2>{});
    x += turned(x, std::integral_constant<int, 4>{});
    x += turned(x, std::integral_constant<int, 8>{});
    return __uint_as_float(across16(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

}  // namespace
}  // namespace flashopt

#endif  // FLASHOPT_FP8_H
