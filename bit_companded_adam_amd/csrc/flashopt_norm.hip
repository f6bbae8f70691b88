// Root-mean-square norm with the residual's addition (flashopt_rms_norm), its
// output in the input's type or in 8 bits with scales, and its backward pass
// (flashopt_rms_norm_backward).
//
//   h = x + residual, rounded to their type       r = 1 / sqrt(mean h^2 + eps)
//   y = (h r) gain, in fp32, rounded once
//   with u = dy gain, t = h r, c = mean(u t):
//   dx = r (u - t c) + dh                          dgain = sum over rows dy t
//
// Squares and their sum are fp64, and r is rounded to fp32 once: bf16 and fp32
// squares leave fp32's range at both ends, and y is then the same three fp32
// roundings whatever the order of the sum.
//
// Each pass reads every row once and is bound by memory.  A group of TPR
// threads takes a row, NV vectors of eight columns to a thread, and keeps it in
// registers between the sum and the output.  With a residual, bf16, 8192 x 4096
// takes 41-44 us to 8 bits (235 MB: 5.5 TB/s) and 42 to bf16 (268 MB: 6.4), its
// backward pass with dh 44 (268 MB: 6.1); 8192 x 2048 23 and 26; one row of 4096
// 3.8 and 5.7, which is latency.  Beyond 16384 columns a backward thread holds
// four vectors of three matrices and spills: 2048 x 16384 takes 59 us (4.6 TB/s),
// 2048 x 20000 101 (3.2).  (Sums over a wavefront by LDS permutations
// instead of DPP, and the gain loaded after the sum, cost the first of these 15
// us; without the next row's loads under way the backward pass takes 58.)

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flashopt.h"
#include "flashopt_fp8.h"
#include "flashopt_internal.h"

namespace flashopt {
namespace {

// Sum over a wavefront, known to all of its lanes (wave_sum in fp64).
__device__ __forceinline__ double wave_sum(double x)
{
    auto halves = [](double v, auto &&f) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = f(static_cast<uint32_t>(b)), hi = f(static_cast<uint32_t>(b >> 32));
        return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
    };
    x += halves(x, [](uint32_t w) { return rotated<1>(w); });
    x += halves(x, [](uint32_t w) { return rotated<2>(w); });
    x += halves(x, [](uint32_t w) { return rotated<4>(w); });
    x += halves(x, [](uint32_t w) { return rotated<8>(w); });
    // (a sum of two does not depend on their order, so each of the pair may
    // take the other's)
    x += halves(x, [](uint32_t w) {
        const auto s = __builtin_amdgcn_permlane16_swap(w, w, false, false);
        return static_cast<uint32_t>((threadIdx.x & 16) ? s[0] : s[1]);
    });
    x += halves(x, [](uint32_t w) {
        const auto s = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        return static_cast<uint32_t>((threadIdx.x & 32) ? s[0] : s[1]);
    });
    return x;
}

// Sum over the TPR threads of a row, known to all of them.  With more than a
// wavefront to a row the workgroup is that row's, and `scratch` (TPR / 64
// values) is free again after the next barrier.
template <int TPR, typename T>
__device__ __forceinline__ T row_sum(T x, T *scratch)
{
    x = wave_sum(x);
    if constexpr (TPR > kWaveLanes) {
        constexpr int kWaves = TPR / kWaveLanes;
        if ((threadIdx.x & (kWaveLanes - 1)) == 0) scratch[threadIdx.x / kWaveLanes] = x;
        __syncthreads();
        x = scratch[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) x += scratch[w];
    }
    return x;
}

struct NormIn {
    const uint8_t *x, *residual, *gain;      // residual: or nullptr
    int64_t x_bytes, residual_bytes;         // of a row's stride
    int64_t rows, cols;
    double eps;
    bool gain_fp32;
};
struct NormOut {
    uint8_t *h, *y, *codes, *scales;         // each, or nullptr
    float *rstd;
    int64_t h_bytes, y_bytes;
    bool e5m2;
};

__device__ __forceinline__ void gains(const uint8_t *gain, bool fp32, int64_t c, int64_t cols, float (&g)[8])
{
    if (fp32) {
        const Eight<true> f = load8<true, false>(gain + c * 4, cols - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = value(f, j);
    } else {
        const Eight<false> f = load8<false, false>(gain + c * 2, cols - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = value(f, j);
    }
}

// Eight normed values to wherever they go: y, and codes under the scale of
// their group's sixteen lanes (values past the row's end are zeros).
template <bool F32>
__device__ __forceinline__ void emit(const NormOut &o, int64_t row, int64_t c, int64_t cols, const float (&v)[8])
{
    if (o.y && c < cols) store8<F32>(o.y + row * o.y_bytes + c * (F32 ? 4 : 2), rounded8<F32>(v), cols - c);
    if (o.codes) {
        const Eight<true> f = rounded8<true>(v);
        const uint32_t top = max16(largest_of(f));
        const uint32_t scale = o.e5m2 ? fp8_scale<kE5M2>(top) : fp8_scale<kE4M3>(top);
        u32x2 q = o.e5m2 ? row_codes<true, kE5M2>(f, scale) : row_codes<true, kE4M3>(f, scale);
        uint32_t b = scale >> 23;
        if (top >= kInfinite) {
            q = u32x2{0u, 0u};
            b = kNanByte;
        }
        if (c < mx_padded(cols)) {
            *reinterpret_cast<u32x2 *>(o.codes + row * mx_padded(cols) + c) = q;
            if ((threadIdx.x & 15) == 0) o.scales[row * fp8_scale_stride(cols) + c / 128] = static_cast<uint8_t>(b);
        }
    }
}

// x + residual in fp32, rounded to their type.
template <bool F32>
__device__ __forceinline__ Eight<F32> added(const Eight<F32> &a, const Eight<F32> &b)
{
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = value(a, j) + value(b, j);
    return rounded8<F32>(v);
}

// NV = 0: a row of any length, read again for the output (h where there is
// one: x otherwise).
template <bool F32, int TPR, int NV>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads)
rms_norm_kernel(NormIn in, NormOut out)
{
    constexpr int kGroup = TPR > kThreads ? TPR : kThreads, kRowsAtOnce = TPR > kWaveLanes ? 1 : kGroup / TPR;
    constexpr int kEsz = F32 ? 4 : 2;
    static_assert(TPR == kWaveLanes || TPR == kGroup, "a wavefront or a workgroup to a row");
    __shared__ double s_sum[2][kGroup / kWaveLanes];
    const int t = threadIdx.x % TPR;
    const int64_t cols = in.cols;
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce + threadIdx.x / TPR; row < in.rows;
         row += static_cast<int64_t>(gridDim.x) * kRowsAtOnce, turn ^= 1) {
        const uint8_t *x = in.x + row * in.x_bytes, *residual = in.residual + row * in.residual_bytes;
        uint8_t *h = out.h + row * out.h_bytes;
        double sum = 0.0;
        Eight<F32> keep[NV > 0 ? NV : 1];
        auto take = [&](int64_t c) {
            Eight<F32> f = load8<F32, false>(x + c * kEsz, cols - c);
            if (in.residual) {
                f = added(f, load8<F32, false>(residual + c * kEsz, cols - c));
                if (c < cols) store8<F32>(h + c * kEsz, f, cols - c);
            }
            return f;
        };
        auto square = [&](const Eight<F32> &f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double v = static_cast<double>(value(f, j));
                sum = __builtin_fma(v, v, sum);
            }
        };
        // a workgroup with one row loads the gain while it waits for the row;
        // wavefronts with a row each have others beside them
        constexpr bool kEarly = TPR > kWaveLanes && NV > 0 && NV < 4;
        float gain[kEarly ? NV : 1][8];
        if constexpr (kEarly) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                gains(in.gain, in.gain_fp32, (static_cast<int64_t>(v) * TPR + t) * 8, cols, gain[v]);
        }
        if constexpr (NV > 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) keep[v] = take((static_cast<int64_t>(v) * TPR + t) * 8);
#pragma unroll
            for (int v = 0; v < NV; ++v) square(keep[v]);
        } else {
            for (int64_t c = t * 8; c < cols; c += TPR * 8) square(take(c));
        }
        sum = row_sum<TPR>(sum, s_sum[turn]);
        const float r = static_cast<float>(1.0 / __builtin_sqrt(sum / static_cast<double>(cols) + in.eps));
        if (out.rstd && t == 0) out.rstd[row] = r;
        if (!out.y && !out.codes) continue;
        auto give = [&](int64_t c, const Eight<F32> &f, int v) {
            float g[8], y[8];
            if constexpr (!kEarly) gains(in.gain, in.gain_fp32, c, cols, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = c + j < cols ? (value(f, j) * r) * (kEarly ? gain[v][j] : g[j]) : 0.0f;
            emit<F32>(out, row, c, cols, y);
        };
        // a group's sixteen lanes take part together, to the end of the padded row
        if constexpr (NV > 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) give((static_cast<int64_t>(v) * TPR + t) * 8, keep[v], v);
        } else {
            const uint8_t *from = in.residual ? h : x;
            for (int64_t c = t * 8; c < mx_padded(cols); c += TPR * 8)
                give(c, load8<F32, false>(from + c * kEsz, cols - c), 0);
        }
        if (out.codes)                        // the rest of the padded row of scales
            for (int64_t i = (cols + 127) / 128 + t; i < fp8_scale_stride(cols); i += TPR)
                out.scales[row * fp8_scale_stride(cols) + i] = 0;
    }
}

// -------------------------------------------------------------- backward

struct GradIn {
    const uint8_t *dy, *dh, *h, *gain;       // dh: or nullptr
    const float *rstd;
    int64_t dy_bytes, dh_bytes, h_bytes;
    int64_t rows, cols;
    bool gain_fp32;
};

// A workgroup takes rows in turn, as the forward pass does, and keeps its
// threads' columns of dgain in registers over all of them; partial[workgroup]
// is added up in order by norm_gain_kernel.  dx is no __restrict__ pointer: it
// may be dy or dh itself.  While a row waits for its sum, the
// next one's loads are under way (kAhead, where registers allow).  DY32: dy is
// fp32, whatever the other matrices are: 8192 x 2048 beside bf16 29.5 us for
// 25.6 with a bf16 dy, 8192 x 4096 63 for 44.
template <bool F32, bool DY32, int TPR, int NV>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads)
rms_norm_backward_kernel(GradIn in, uint8_t *dx, int64_t dx_bytes, float *__restrict__ partial)
{
    constexpr int kGroup = TPR > kThreads ? TPR : kThreads, kRowsAtOnce = TPR > kWaveLanes ? 1 : kGroup / TPR;
    constexpr int kEsz = F32 ? 4 : 2, kDyEsz = DY32 ? 4 : 2;
    constexpr bool kAhead = NV * (F32 ? 2 : 1) <= 2 && TPR < 1024;
    constexpr bool kLdsGain = NV >= 4;       // the columns of dgain of that many vectors go to LDS, each thread's its own
    __shared__ float s_dgain[kLdsGain ? NV * 8 : 1][kLdsGain ? TPR : 1];
    __shared__ float s_sum[2][kGroup / kWaveLanes];
    __shared__ float s_gain[kRowsAtOnce > 1 ? kRowsAtOnce * TPR * 8 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t cols = in.cols;
    auto column = [&](int v) { return (static_cast<int64_t>(v) * TPR + t) * 8; };
    struct Row {
        Eight<DY32> dy[NV];
        Eight<F32> h[NV], dh[kAhead ? NV : 1];
        float r;
    };
    auto load_dh = [&](int64_t row, int64_t c) {
        if (!dx || !in.dh) return Eight<F32>{};
        return load8<F32, false>(in.dh + row * in.dh_bytes + c * kEsz, cols - c);
    };
    auto load = [&](Row &x, int64_t row) {
        x.r = in.rstd[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = column(v);
            x.dy[v] = load8<DY32, false>(in.dy + row * in.dy_bytes + c * kDyEsz, cols - c);
            x.h[v] = load8<F32, false>(in.h + row * in.h_bytes + c * kEsz, cols - c);
            if constexpr (kAhead) x.dh[v] = load_dh(row, c);
        }
    };
    float gain[kAhead ? NV : 1][8];
    if constexpr (kAhead) {
#pragma unroll
        for (int v = 0; v < NV; ++v) gains(in.gain, in.gain_fp32, column(v), cols, gain[v]);
    }
    float dgain[kLdsGain ? 1 : NV][8];
    auto gain_sum = [&](int v, int j) -> float & {
        if constexpr (kLdsGain) return s_dgain[v * 8 + j][t];
        else return dgain[v][j];
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) gain_sum(v, j) = 0.0f;
    const int64_t hop = static_cast<int64_t>(gridDim.x) * kRowsAtOnce;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce + threadIdx.x / TPR;
    Row now, next;
    if (kAhead && row < in.rows) load(next, row);
    for (int turn = 0; row < in.rows; row += hop, turn ^= 1) {
        if constexpr (kAhead) {
            now = next;
            if (row + hop < in.rows) load(next, row + hop);
        } else {
            load(now, row);
        }
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float g[8];
            if constexpr (!kAhead) gains(in.gain, in.gain_fp32, column(v), cols, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = value(now.dy[v], j), x = value(now.h[v], j) * now.r;
                gain_sum(v, j) = __builtin_fmaf(d, x, gain_sum(v, j));
                sum = __builtin_fmaf(d * (kAhead ? gain[v][j] : g[j]), x, sum);
            }
        }
        if (!dx) continue;
        const float c1 = row_sum<TPR>(sum, s_sum[turn]) / static_cast<float>(cols);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = column(v);
            if (c >= cols) continue;
            float g[8], o[8];
            if constexpr (!kAhead) gains(in.gain, in.gain_fp32, c, cols, g);
            const Eight<F32> dh = kAhead ? now.dh[kAhead ? v : 0] : load_dh(row, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = value(now.dy[v], j) * (kAhead ? gain[v][j] : g[j]);
                o[j] = now.r * (u - (value(now.h[v], j) * now.r) * c1) + value(dh, j);
            }
            store8<F32>(dx + row * dx_bytes + c * kEsz, rounded8<F32>(o), cols - c);
        }
    }
    if (!partial) return;
    float *p = partial + static_cast<int64_t>(blockIdx.x) * cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = column(v);
        if constexpr (kRowsAtOnce > 1) {      // the wavefronts' sums, in their order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) s_gain[(threadIdx.x / TPR * 8 + j) * TPR + t] = gain_sum(v, j);
            __syncthreads();
            if (threadIdx.x < TPR) {
#pragma unroll
                for (int w = 1; w < kRowsAtOnce; ++w)
#pragma unroll
                    for (int j = 0; j < 8; ++j) gain_sum(v, j) += s_gain[(w * 8 + j) * TPR + t];
            }
        }
        if (kRowsAtOnce == 1 || threadIdx.x < TPR) {
            Eight<true> f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f.w[j] = __float_as_uint(gain_sum(v, j));
            store8<true>(reinterpret_cast<uint8_t *>(p + c), f, cols - c);
        }
    }
}

// dgain = the sum of the partial rows, in fp64 and in an order of their number
// alone; 32 columns to a workgroup, 32 threads to a column.
constexpr int kGainCols = 32, kGainThreads = 1024, kGainShares = kGainThreads / kGainCols;
__global__ void __launch_bounds__(kGainThreads)
norm_gain_kernel(const float *__restrict__ partial, int count, int64_t cols, uint8_t *__restrict__ dgain, bool fp32)
{
    __shared__ double s_sum[kGainShares][kGainCols];
    const int col = threadIdx.x % kGainCols, share = threadIdx.x / kGainCols;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kGainCols + col;
    double sum = 0.0;
    if (c < cols) {
#pragma unroll 4
        for (int i = share; i < count; i += kGainShares) sum += static_cast<double>(partial[i * cols + c]);
    }
    s_sum[share][col] = sum;
    __syncthreads();
    if (share == 0 && c < cols) {
#pragma unroll
        for (int w = 1; w < kGainShares; ++w) sum += s_sum[w][col];
        if (fp32) reinterpret_cast<float *>(dgain)[c] = static_cast<float>(sum);
        else reinterpret_cast<uint16_t *>(dgain)[c] = bf16_rne(static_cast<float>(sum));
    }
}

// ------------------------------------------------------------- launching

// The launch for rows of so many columns: f(TPR, NV), a wavefront or the
// smallest workgroup whose registers hold a row.  Rows x columns in us, forward
// to 8 bits / backward: 8192 x 1024 by wavefronts (64, 2) 15.0 / 17.3, by (256, 1)
// 20.3 / 21.6; 8192 x 2048 (256, 1) 23.7 / 25.9, (64, 4) 26.6 / 34.0; 8192 x 4096
// (256, 2) 41.6 / 45.6, (512, 1) 43.5 / 44.1, (64, 8) 53.0 / -; one row of 4096
// (256, 2) 4.8 / 6.3, (512, 1) 3.9 / 5.7, (1024, 1) 4.4 / 7.5; 4096 x 8192 (512, 2)
// 46.3 / 45.2, (256, 4) 48.1 / 64.7.
template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
hipError_t by_columns(int64_t cols, F &&f)
{
    if (cols <= 512) return f(Int<64>{}, Int<1>{});
    if (cols <= 1024) return f(Int<64>{}, Int<2>{});
    if (cols <= 2048) return f(Int<256>{}, Int<1>{});
    if (cols <= 4096) return f(Int<512>{}, Int<1>{});
    if (cols <= 8192) return f(Int<512>{}, Int<2>{});
    if (cols <= 16384) return f(Int<1024>{}, Int<2>{});
    if (cols <= 32768) return f(Int<1024>{}, Int<4>{});
    return f(Int<1024>{}, Int<0>{});
}

template <int TPR>
unsigned row_groups(int64_t rows)
{
    return static_cast<unsigned>(TPR > kWaveLanes ? rows : (rows + kThreads / TPR - 1) / (kThreads / TPR));
}

// Workgroups of a backward pass: two to a CU, one of 512 threads or more (with
// two, 8192 x 8192 takes 50.0 us instead of 45.2, for the partial rows).
template <int TPR>
unsigned backward_groups(int64_t rows)
{
    constexpr unsigned kMost = TPR >= 512 ? kCus : 2 * kCus;
    const unsigned groups = row_groups<TPR>(rows);
    return groups < kMost ? groups : kMost;
}

template <bool F32>
hipError_t norm_type(const NormIn &in, const NormOut &out, hipStream_t st)
{
    return by_columns(in.cols, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const unsigned groups = row_groups<TPR>(in.rows);
        hipLaunchKernelGGL((rms_norm_kernel<F32, TPR, NV>), dim3(groups < (1u << 20) ? groups : (1u << 20)),
                           dim3(TPR > kThreads ? TPR : kThreads), 0, st, in, out);
        return hipGetLastError();
    });
}

template <bool F32, bool DY32>
hipError_t backward_type(const GradIn &in, uint8_t *dx, int64_t dx_bytes, uint8_t *dgain, float *partial,
                         hipStream_t st)
{
    return by_columns(in.cols, [&](auto tpr, auto nv) -> hipError_t {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        if constexpr (NV == 0) {
            return hipErrorInvalidValue;
        } else {
            const unsigned grid = backward_groups<TPR>(in.rows);
            if (grid > 0) {
                hipLaunchKernelGGL((rms_norm_backward_kernel<F32, DY32, TPR, NV>), dim3(grid),
                                   dim3(TPR > kThreads ? TPR : kThreads), 0, st, in, dx, dx_bytes, partial);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess || !dgain) return e;
            }
            hipLaunchKernelGGL(norm_gain_kernel, dim3(static_cast<unsigned>((in.cols + kGainCols - 1) / kGainCols)),
                               dim3(kGainThreads), 0, st, partial, static_cast<int>(grid), in.cols, dgain,
                               in.gain_fp32);
            return hipGetLastError();
        }
    });
}

}  // namespace

int64_t norm_grad_partials(int64_t rows, int64_t cols)
{
    int64_t most = 0;
    auto with = [&](int64_t c) {
        (void)by_columns(c, [&](auto tpr, auto) {
            const int64_t size = backward_groups<decltype(tpr)::value>(rows) * c;
            most = size > most ? size : most;
            return hipSuccess;
        });
    };
    // a narrower pass may have more workgroups: the widest of each of by_columns'
    for (int64_t c : {512, 1024, 2048, 4096, 8192, 16384, 32768})
        if (c < cols) with(c);
    with(cols);
    return most;
}

hipError_t launch_rms_norm(const NormCall &n, hipStream_t st)
{
    const int esz = n.x.fp32 ? 4 : 2;
    const NormIn in{static_cast<const uint8_t *>(n.x.data), static_cast<const uint8_t *>(n.residual.data),
                    static_cast<const uint8_t *>(n.gain), n.x.row_stride * esz, n.residual.row_stride * esz,
                    n.x.rows, n.x.cols, n.eps, n.gain_fp32};
    // codes along columns need the statistics of 128 rows first: then both
    // layouts come from a second launch, which reads h again
    const bool tiles = n.q.codes_t != nullptr;
    const NormOut out{static_cast<uint8_t *>(n.h.data), static_cast<uint8_t *>(n.y.data),
                      tiles ? nullptr : n.q.codes, n.q.scales, n.rstd, n.h.row_stride * esz, n.y.row_stride * esz,
                      n.format == kE5M2};
    hipError_t e = n.x.fp32 ? norm_type<true>(in, out, st) : norm_type<false>(in, out, st);
    if (e != hipSuccess || !tiles) return e;
    return launch_fp8_normed(n.residual.data ? n.h : n.x, n.rstd, n.gain, n.gain_fp32, n.format, n.q, st);
}

hipError_t launch_rms_norm_backward(const NormGradCall &n, hipStream_t st)
{
    const int esz = n.h.fp32 ? 4 : 2;
    const GradIn in{static_cast<const uint8_t *>(n.dy.data), static_cast<const uint8_t *>(n.dh.data),
                    static_cast<const uint8_t *>(n.h.data), static_cast<const uint8_t *>(n.gain), n.rstd,
                    n.dy.row_stride * (n.dy.fp32 ? 4 : 2), n.dh.row_stride * esz, n.h.row_stride * esz, n.h.rows, n.h.cols,
                    n.gain_fp32};
    uint8_t *dx = static_cast<uint8_t *>(n.dx.data), *dgain = static_cast<uint8_t *>(n.dgain);
    float *partial = dgain ? n.partial : nullptr;
    const int64_t dx_bytes = n.dx.row_stride * esz;
    if (n.h.fp32) return backward_type<true, true>(in, dx, dx_bytes, dgain, partial, st);
    return n.dy.fp32 ? backward_type<false, true>(in, dx, dx_bytes, dgain, partial, st)
                     : backward_type<false, false>(in, dx, dx_bytes, dgain, partial, st);
}

}  // namespace flashopt
