// The global gradient norm over a list of tensors, and clipping by it
// (flashopt_grad_norm, flashopt_grad_clip).
//
//   norm  = sqrt(sum over tensors and elements of g^2)
//   scale = min(1, max_norm / (norm + 1e-6))
//   clip:  g <- g * scale, one fp32 product rounded to g's own type
//
// Sums: every square and every sum is fp64.  bf16 and fp32 both reach 2^127,
// whose square overflows fp32, and 2^-100, whose square vanishes in it; in
// fp64 neither happens and a sum of 2^40 terms still carries 40 bits.  norm
// and scale are rounded to fp32 once, at the end.  Per element that is one
// conversion and one fp64 fma, about a tenth of the VALU's fp64 rate at the
// rate the memory delivers bf16 gradients, so the norm stays bound by HBM.
//
// Order: a launch of B workgroups gives workgroup b the chunks
// [b total / B, (b + 1) total / B) of the list and stores one partial sum for
// it; the workgroup that finishes last adds the B partials in index order.
// Who is last varies, what it adds does not: the result depends on the list
// and on B alone, never on timing, and there are no floating-point atomics.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flashopt.h"
#include "flashopt_internal.h"

namespace flashopt {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) const u32x4 g_cu4;
typedef __attribute__((address_space(1))) u32x4 g_u4;

constexpr int kNormThreads = 1024;
constexpr int kScaleThreads = kBlockThreads;

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// fp32 -> bf16, round to nearest even; a NaN keeps its upper half, made quiet.
__device__ __forceinline__ uint32_t bf16_rne(float x)
{
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// The list's descriptors: in the kernel arguments for a short list, in the
// staged table for a long one.
struct ListArgs {
    GradDesc desc[kGradArgTensors];
    int32_t start[kGradArgTensors + 1];
};

struct ListTable {
    const GradDesc *desc;
    const int32_t *start;
};

__device__ __forceinline__ GradDesc list_desc(const ListArgs &l, int t) { return l.desc[t]; }
__device__ __forceinline__ GradDesc list_desc(const ListTable &l, int t) { return l.desc[t]; }
__device__ __forceinline__ int32_t list_start(const ListArgs &l, int t) { return l.start[t]; }
__device__ __forceinline__ int32_t list_start(const ListTable &l, int t) { return l.start[t]; }

// The tensor that owns chunk c: the last one whose first chunk is <= c.
template <typename List>
__device__ __forceinline__ int tensor_of(const List &list, int n_tensors, int32_t c)
{
    int lo = 0, hi = n_tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list_start(list, mid) <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls segment(desc, first element, element count) for the parts of the
// tensors that chunks [c0, c1) cover, in order; everything here is uniform
// across the workgroup.
template <typename List, typename Segment>
__device__ __forceinline__ void for_segments(const List &list, int n_tensors, int32_t c0, int32_t c1,
                                             Segment &&segment)
{
    if (c0 >= c1) return;
    for (int t = tensor_of(list, n_tensors, c0); t < n_tensors; ++t) {
        const int32_t s = list_start(list, t), e = list_start(list, t + 1);
        if (s >= c1) break;
        const GradDesc d = list_desc(list, t);
        const int32_t a = s > c0 ? s : c0, b = e < c1 ? e : c1;
        if (a >= b) continue;                     // an empty tensor
        const int64_t first = static_cast<int64_t>(a - s) * kGradChunk;
        int64_t last = static_cast<int64_t>(b - s) * kGradChunk;
        if (last > d.numel) last = d.numel;
        segment(d, first, last - first);
    }
}

// Elements before the first 16-byte boundary at p (the pointer is aligned to
// its element, not necessarily to 16 bytes), at most n.
template <int ESZ>
__device__ __forceinline__ int64_t head_elems(const void *p, int64_t n)
{
    const int64_t h = static_cast<int64_t>((0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p))) & 15u) / ESZ;
    return h < n ? h : n;
}

template <int ESZ>
__device__ __forceinline__ float elem(const uint8_t *p, int64_t i)
{
    if constexpr (ESZ == 4) return reinterpret_cast<const float *>(p)[i];
    else return bf16_value(reinterpret_cast<const uint16_t *>(p)[i]);
}

__device__ __forceinline__ void add_square(double &acc, float x)
{
    const double d = x;
    acc = __builtin_fma(d, d, acc);
}

template <int ESZ>
__device__ __forceinline__ void add_vector(double (&acc)[2], u32x4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (ESZ == 4) {
            add_square(acc[k & 1], __uint_as_float(w[k]));
        } else {
            add_square(acc[0], __uint_as_float(w[k] << 16));
            add_square(acc[1], __uint_as_float(w[k] & 0xFFFF0000u));
        }
    }
}

// Every gradient is read once, or read and written once, by these kernels:
// nontemporal accesses (the norm of 2.4 GB runs at 6.45 TB/s with them and 5.90
// without; the scaling's reads and writes keep 6.2 TB/s of both ways).
__device__ __forceinline__ u32x4 load16(const uint8_t *p, int64_t i)
{
    return __builtin_nontemporal_load((g_cu4 *)p + i);
}
__device__ __forceinline__ void store16(uint8_t *p, int64_t i, u32x4 v)
{
    __builtin_nontemporal_store(v, (g_u4 *)p + i);
}

// This thread's share of the sum of squares of n elements at p: 16-byte
// loads, kDepth of them in flight, the elements outside whole 16-byte words
// one by one.
template <int ESZ>
__device__ __forceinline__ void add_segment(double (&acc)[2], const uint8_t *p, int64_t n)
{
    constexpr int kDepth = 4;
    const int tid = threadIdx.x;
    const int64_t head = head_elems<ESZ>(p, n);
    if (tid < head) add_square(acc[0], elem<ESZ>(p, tid));
    const uint8_t *q = p + head * ESZ;
    const int64_t words = (n - head) * ESZ / 16;
    int64_t i = tid;
    for (; i + (kDepth - 1) * kNormThreads < words; i += kDepth * kNormThreads) {
        u32x4 v[kDepth];
#pragma unroll
        for (int k = 0; k < kDepth; ++k) v[k] = load16(q, i + k * kNormThreads);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) add_vector<ESZ>(acc, v[k]);
    }
    for (; i < words; i += kNormThreads) add_vector<ESZ>(acc, load16(q, i));
    const int64_t done = head + words * (16 / ESZ);
    if (tid < n - done) add_square(acc[1], elem<ESZ>(p, done + tid));
}

// Sum over the workgroup, in a fixed order; the result on thread 0.
__device__ __forceinline__ double block_sum(double x, double *s_wave)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, kWaveLanes);
    __syncthreads();
    if ((threadIdx.x & (kWaveLanes - 1)) == 0) s_wave[threadIdx.x / kWaveLanes] = x;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kNormThreads / kWaveLanes; ++w) t += s_wave[w];
    return t;
}

__device__ __forceinline__ int32_t share(int32_t total, uint32_t b, uint32_t nb)
{
    return static_cast<int32_t>(static_cast<int64_t>(total) * b / nb);
}

// A list of 1.2e9 bf16 elements takes 371 us (6.45 TB/s), one of 2.2e8 67 us
// (6.47); memory bounds it, a large copy reaching 6.2 and bare reads 6.9.
template <typename List>
__global__ void __launch_bounds__(kNormThreads)
grad_norm_kernel(List list, int n_tensors, int32_t total_chunks, double max_norm,
                 GradSums *__restrict__ sums, float *__restrict__ out)
{
    __shared__ double s_wave[kNormThreads / kWaveLanes];
    __shared__ bool s_last;
    const uint32_t nb = gridDim.x, b = blockIdx.x;
    double acc[2] = {0.0, 0.0};
    for_segments(list, n_tensors, share(total_chunks, b, nb), share(total_chunks, b + 1, nb),
                 [&](const GradDesc &d, int64_t first, int64_t n) {
                     const uint8_t *p = static_cast<const uint8_t *>(d.data);
                     if (d.fp32) add_segment<4>(acc, p + first * 4, n);
                     else add_segment<2>(acc, p + first * 2, n);
                 });
    double total = block_sum(acc[0] + acc[1], s_wave);
    if (nb > 1) {
        if (threadIdx.x == 0) {
            // Partials and counter are touched by agent-scope atomics alone,
            // which act at the memory all XCDs share, and the exchange's
            // returned value is waited for before the counter moves: whoever
            // reads the last count finds every partial.  (A fence would
            // write back and drop the XCD's whole L2 for each workgroup:
            // 95 us on a launch of 2048.)
            const uint64_t old = __hip_atomic_exchange(
                reinterpret_cast<uint64_t *>(&sums->partial[b]), __builtin_bit_cast(uint64_t, total),
                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" : : "v"(old) : "memory");
            // the count wraps to zero with the last workgroup, ready for the
            // next launch
            s_last = atomicInc(&sums->finished, nb - 1) == nb - 1;
        }
        __syncthreads();
        if (!s_last) return;
        double x = 0.0;
        for (uint32_t i = threadIdx.x; i < nb; i += kNormThreads)
            x += __hip_atomic_load(&sums->partial[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        total = block_sum(x, s_wave);
    }
    if (threadIdx.x == 0) {
        const double norm = sqrt(total);
        const double scale = max_norm / (norm + 1e-6);
        out[0] = static_cast<float>(norm);
        out[1] = scale > 1.0 ? 1.0f : static_cast<float>(scale);   // a NaN norm gives a NaN scale
    }
}

template <int ESZ>
__device__ __forceinline__ u32x4 scaled_vector(u32x4 v, float s)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (ESZ == 4) {
            w[k] = __float_as_uint(__uint_as_float(w[k]) * s);
        } else {
            const uint32_t lo = bf16_rne(__uint_as_float(w[k] << 16) * s);
            const uint32_t hi = bf16_rne(__uint_as_float(w[k] & 0xFFFF0000u) * s);
            w[k] = lo | (hi << 16);
        }
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <int ESZ>
__device__ __forceinline__ void scale_elem(uint8_t *p, int64_t i, float s)
{
    if constexpr (ESZ == 4) reinterpret_cast<float *>(p)[i] *= s;
    else reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(bf16_rne(elem<2>(p, i) * s));
}

template <int ESZ>
__device__ __forceinline__ void scale_segment(uint8_t *p, int64_t n, float s)
{
    constexpr int kDepth = 4;
    const int tid = threadIdx.x;
    const int64_t head = head_elems<ESZ>(p, n);
    if (tid < head) scale_elem<ESZ>(p, tid, s);
    uint8_t *q = p + head * ESZ;
    const int64_t words = (n - head) * ESZ / 16;
    int64_t i = tid;
    for (; i + (kDepth - 1) * kScaleThreads < words; i += kDepth * kScaleThreads) {
        u32x4 v[kDepth];
#pragma unroll
        for (int k = 0; k < kDepth; ++k) v[k] = load16(q, i + k * kScaleThreads);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) store16(q, i + k * kScaleThreads, scaled_vector<ESZ>(v[k], s));
    }
    for (; i < words; i += kScaleThreads) store16(q, i, scaled_vector<ESZ>(load16(q, i), s));
    const int64_t done = head + words * (16 / ESZ);
    if (tid < n - done) scale_elem<ESZ>(p, done + tid, s);
}

// g <- g * scale over the list.  A scale of exactly 1 changes no value (the
// product is exact and a bf16 value rounds to itself), so the gradients are
// neither read nor written then.  A workgroup takes one chunk at a time, the
// grid's neighbours taking its neighbours: 13-17% faster than contiguous
// ranges of chunks, which the read-only norm does not mind (1%) and which
// save it the search for each chunk's tensor.
template <typename List>
__global__ void __launch_bounds__(kScaleThreads)
grad_scale_kernel(List list, int n_tensors, int32_t total_chunks, const float *__restrict__ scale)
{
    const float s = *scale;
    if (s == 1.0f) return;
    for (uint32_t u = blockIdx.x; u < static_cast<uint32_t>(total_chunks); u += gridDim.x) {
        const int32_t c = static_cast<int32_t>(u);
        const int t = tensor_of(list, n_tensors, c);
        const GradDesc d = list_desc(list, t);
        const int64_t first = static_cast<int64_t>(c - list_start(list, t)) * kGradChunk;
        const int64_t n = d.numel - first < kGradChunk ? d.numel - first : kGradChunk;
        uint8_t *p = static_cast<uint8_t *>(d.data);
        if (d.fp32) scale_segment<4>(p + first * 4, n, s);
        else scale_segment<2>(p + first * 2, n, s);
    }
}

// An empty list (or one of empty tensors): norm 0.
__global__ void grad_empty_kernel(double max_norm, float *out)
{
    const double scale = max_norm / 1e-6;
    out[0] = 0.0f;
    out[1] = scale > 1.0 ? 1.0f : static_cast<float>(scale);
}

// Workgroups of a scaling at most (a dispatch counts work-items in 32 bits).
constexpr int kScaleGrid = 1 << 20;

unsigned grid_of(int32_t total_chunks, int most)
{
    return static_cast<unsigned>(total_chunks < most ? total_chunks : most);
}

template <typename List>
hipError_t launch(const List &list, int n, int32_t total, double max_norm, bool clip, GradSums *sums,
                  float *out, hipStream_t st)
{
    hipLaunchKernelGGL(grad_norm_kernel<List>, dim3(grid_of(total, kGradPartials)), dim3(kNormThreads), 0,
                       st, list, n, total, max_norm, sums, out);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !clip) return e;
    hipLaunchKernelGGL(grad_scale_kernel<List>, dim3(grid_of(total, kScaleGrid)), dim3(kScaleThreads), 0,
                       st, list, n, total, out + 1);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_args(const GradDesc *desc, const int32_t *start, int n, int32_t total,
                            double max_norm, bool clip, GradSums *sums, float *out, hipStream_t st)
{
    ListArgs list{};
    for (int i = 0; i < n; ++i) {
        list.desc[i] = desc[i];
        list.start[i] = start[i];
    }
    list.start[n] = total;
    return launch(list, n, total, max_norm, clip, sums, out, st);
}

hipError_t launch_grad_table(const GradDesc *desc, const int32_t *start, int n, int32_t total,
                             double max_norm, bool clip, GradSums *sums, float *out, hipStream_t st)
{
    return launch(ListTable{desc, start}, n, total, max_norm, clip, sums, out, st);
}

hipError_t launch_grad_empty(double max_norm, float *out, hipStream_t st)
{
    hipLaunchKernelGGL(grad_empty_kernel, dim3(1), dim3(1), 0, st, max_norm, out);
    return hipGetLastError();
}

}  // namespace flashopt
