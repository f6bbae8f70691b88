// Internal declarations shared by the kernels (flashopt_kernels.hip) and the
// C-ABI host layer (flashopt_api.cpp) of libflashopt.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flashopt {

// Work decomposition: 1024-element chunks, 16 elements per lane of a
// 64-lane wavefront, processed in units of consecutive elements (the step
// kernels give each wavefront one unit, see the kernels); quantization
// groups are 32 elements; a 256-thread workgroup runs four wavefronts.
constexpr int kLaneElems = 16;
constexpr int kWaveLanes = 64;
constexpr int kChunkElems = kLaneElems * kWaveLanes;   // 1024
constexpr int kBlockThreads = 256;
constexpr int kGroup = 32;

// State storage of the step: codes with fp16 group scales under the linear or
// the companded specs, or plain fp32 moments (the unquantized-states ablation).
enum : int { kStatesLinear = 0, kStatesCompanded = 1, kStatesFp32 = 2 };

// The step kernels' parameter formats, as their master-bits argument: 24 and
// 32 split a bf16 parameter with int8 / int16 rho, 0 updates a bf16
// parameter without a split, kParamF32 updates an fp32 parameter (with an
// fp32 gradient) in place, never split.
constexpr int kParamF32 = 1;

// Per-tensor descriptor of the multi-tensor step, staged in the workspace.
// With fp32 states m_codes / v_codes point to float arrays.
struct DevTensor {
    uint16_t *param;
    const uint16_t *grad;
    void *rho;
    int8_t *m_codes;
    uint16_t *m_scales;
    uint8_t *v_codes;
    uint16_t *v_scales;
    int64_t numel;
};
static_assert(sizeof(DevTensor) == 64, "descriptor layout");

// Byte offsets of a chunk's state in the blocked state layout (bytes = 0:
// the per-tensor streams): block c of a tensor starts at rho + c * bytes and
// holds rho at 0, the m codes at m, the v codes at v, the m scales at ms and
// the v scales at vs.
struct StateLayout {
    uint32_t bytes, m, v, ms, vs;
};

// Scalars of one step.  The fp32 ones are formed in double on the host and
// rounded once (a Python float meeting a float32 tensor); rbc1 and inv_bc2s
// serve the kernel's exact short routes for the bias-correction quotients
// (div_markstein with rbc1; sqrt_quot_x2p32 with inv_bc2s).
struct StepScalars {
    double inv_bc2s;    // 2^64 / bc2 in double: vhat 2^64 inside sqrt_quot_x2p32
    float cwd;          // 1 - lr * wd
    float b1;           // beta1
    float c1;           // 1 - beta1
    float b2;           // beta2
    float c2;           // 1 - beta2
    float bc1;          // 1 - beta1^t
    float bc2;          // 1 - beta2^t
    float lr;
    float eps;
    float lr2;          // lr 2^32 (exact): the numerator's scale on the short route
    float eps2;         // eps 2^32 (exact): the denominator's scale on the short route
    float rbc1;         // 1 / bc1 correctly rounded to fp32
    float kv;           // 255 sqrt(bc2) 2^-32: the variance codes' factor from sqrt(vhat) 2^32
    float m1_max;       // |m1| up to this keeps |lr mhat 2^32| <= 2^100 eps2 and |m1| <= 2^99 bc1
    uint32_t v1_bound;  // v1 bit patterns below this keep vhat below 2^63
    uint32_t num_key;   // (pattern << 1) - 1 of the smallest nonzero |lr mhat 2^32| allowed
    int fast;           // 1 when eps and lr keep the short routes exact (see adamw_scalars)
    int unit_bc;        // bit 0: bc1 is exactly 1, bit 1: bc2 is exactly 1 (later in training)
    StateLayout blk;    // the state layout
    float gs;           // the value at grad_scale, which the kernels fill in
    const float *grad_scale;   // device factor on every gradient, or NULL
};
// The list step kernels (AdamW and FlashSGD) read their scalars from device
// memory: a block of kScalarsBytes at the start of the staged table (the
// workspace, the allocation-free scratch array or a caller's plan), written
// by the same host-to-device copy as the table or by a later one, so that a
// launch can be captured once and replayed with new scalars.
constexpr size_t kScalarsBytes = 128;
static_assert(sizeof(StepScalars) <= kScalarsBytes, "scalar block");
// fp32 scalars of one FlashSGD step (SGD with momentum), formed in double
// on the host and rounded once.
struct SgdScalars {
    float lr;
    float mu;       // momentum
    float cd;       // 1 - dampening
    float wd;       // coupled weight decay
    int has_wd;     // weight_decay != 0
    int first;      // step == 1: the buffer is set to the gradient
    int nesterov;
    StateLayout blk;    // the state layout (no v parts)
    float gs;           // as in StepScalars
    const float *grad_scale;
};
static_assert(sizeof(SgdScalars) <= kScalarsBytes, "scalar block");

// Allocation-free list step: its scalar block and chunk table (up to
// kScratchTensors descriptors, then their chunk starts) live in a device
// array of the library, kScratchBytes long.  scratch_address returns that
// array's address on the current device (looked up once per device).
constexpr int kScratchTensors = 1024;
constexpr size_t kScratchBytes =
    (kScalarsBytes + sizeof(DevTensor) * kScratchTensors + sizeof(int32_t) * (kScratchTensors + 1) + 255) &
    ~size_t(255);
hipError_t scratch_address(void **ptr);

hipError_t launch_quantize(const float *x, int64_t n, unsigned spec, void *codes,
                           uint16_t *scales, hipStream_t stream);
hipError_t launch_dequantize(const void *codes, const uint16_t *scales, int64_t n,
                             unsigned spec, float *out, hipStream_t stream);
hipError_t launch_split(const float *master, int64_t n, int master_bits,
                        uint16_t *param, void *rho, hipStream_t stream);
hipError_t launch_reconstruct(const uint16_t *param, const void *rho, int64_t n,
                              int master_bits, float *master, hipStream_t stream);
// scalars / tensors / chunk_start are device pointers into the staged
// table; chunk_start has n_tensors + 1 entries.  master_bits: 24 | 32 | 0
// (no split) | kParamF32 (AdamW only); states: one of kStates*; scaled: the
// scalars hold a grad_scale.
hipError_t launch_adamw_step(const StepScalars *scalars, const DevTensor *tensors,
                             const int32_t *chunk_start, int n_tensors, int32_t total_chunks,
                             int master_bits, int states, bool scaled, hipStream_t stream);
hipError_t launch_sgd_step(const SgdScalars *scalars, const DevTensor *tensors,
                           const int32_t *chunk_start, int n_tensors, int32_t total_chunks,
                           int master_bits, int states, bool scaled, hipStream_t stream);
// One tensor, its descriptor passed in the kernel arguments (no workspace).
hipError_t launch_adamw_tensor(const DevTensor &d, const StepScalars &sc, int master_bits,
                               int states, hipStream_t stream);
hipError_t launch_sgd_tensor(const DevTensor &d, const SgdScalars &sc, int master_bits,
                             int states, hipStream_t stream);


// ---- gradient norm and clipping (flashopt_grad.hip)

// One gradient of a list; the chunk table counts kGradChunk elements (four or
// eight 16-byte loads of each of a scaling workgroup's 256 threads).
struct GradDesc {
    void *data;
    int64_t numel;
    int32_t fp32;      // 0: bf16, 1: fp32
    int32_t pad;
};
static_assert(sizeof(GradDesc) == 24, "descriptor layout");
constexpr int kGradChunk = 8192;
// Workgroups of a norm at most: two of 1024 threads to a CU, which all run at
// once.  Fewer and larger, because each ends in two atomics that take turns.
constexpr int kGradPartials = 512;
// Lists up to this length travel in the kernel arguments.
constexpr int kGradArgTensors = 64;

// The head of a norm's workspace or plan: how many workgroups of the launch
// in flight have stored their partial sum (zero between launches), and the
// partial sums.
struct GradSums {
    uint32_t finished;
    uint32_t pad[31];
    double partial[kGradPartials];
};
static_assert(sizeof(GradSums) % 128 == 0, "table alignment");

hipError_t launch_grad_args(const GradDesc *desc, const int32_t *start, int n, int32_t total,
                            double max_norm, bool clip, GradSums *sums, float *out, hipStream_t st);
hipError_t launch_grad_table(const GradDesc *desc, const int32_t *start, int n, int32_t total,
                             double max_norm, bool clip, GradSums *sums, float *out, hipStream_t st);
hipError_t launch_grad_empty(double max_norm, float *out, hipStream_t st);

// ---- MXFP4 (flashopt_mx.hip)

// Elements of a padded row.
__host__ __device__ inline int64_t mx_padded(int64_t cols) { return (cols + 127) / 128 * 128; }

// A plain row-major matrix, its rows row_stride elements apart.
struct MxMatrix {
    void *data;
    int64_t rows, cols, row_stride;
    bool fp32;         // or bf16
};

hipError_t launch_mx_quantize(const MxMatrix &x, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                              uint8_t *scales_t, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, const MxMatrix &out,
                                hipStream_t stream);
// x w^T in one launch, x quantized inside it: whether x (a few aligned rows of
// bf16) and the n rows of w allow it, and the launch.
bool mx_linear_direct(const MxMatrix &x, int64_t n);
hipError_t launch_mx_linear_direct(const MxMatrix &x, const uint8_t *w_codes, const uint8_t *w_scales,
                                   const MxMatrix &out, hipStream_t stream);
// out = A B^T with A of out.rows and B of out.cols rows.
hipError_t launch_mx_product(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                             const uint8_t *b_scales, int64_t inner, const MxMatrix &out,
                             hipStream_t stream);

// ---- 8-bit matrices (flashopt_fp8.hip) and the norm (flashopt_norm.hip)

// Formats of codes, as the matrix instructions number them.
constexpr int kE4M3 = 0, kE5M2 = 1;

// Bytes of a row of scales: one for each 128 elements, padded to a multiple of
// 16.  (Rows of codes are mx_padded(cols) bytes.)
__host__ __device__ inline int64_t fp8_scale_stride(int64_t cols) { return (cols + 2047) / 2048 * 16; }

// A quantization's outputs: along rows, of the transpose, or both.
struct Fp8Out {
    uint8_t *codes, *scales, *codes_t, *scales_t;
};

hipError_t launch_fp8_quantize(const MxMatrix &x, int format, bool block, const Fp8Out &q, hipStream_t stream);
// Of (h rstd) gain, both layouts or the transpose.
hipError_t launch_fp8_normed(const MxMatrix &h, const float *rstd, const void *gain, bool gain_fp32, int format,
                             const Fp8Out &q, hipStream_t stream);
hipError_t launch_fp8_dequantize(const uint8_t *codes, const uint8_t *scales, int format, const MxMatrix &out,
                                 hipStream_t stream);
// out = A B^T with A of out.rows and B of out.cols rows; B is E4M3.
hipError_t launch_fp8_product(const uint8_t *a_codes, const uint8_t *a_scales, int a_format, const uint8_t *b_codes,
                              const uint8_t *b_scales, int64_t inner, const MxMatrix &out, hipStream_t stream);

// x w^T in one launch, x quantized inside it: whether x (one row of bf16) allows
// it, and the launch.
bool fp8_linear_direct(const MxMatrix &x);
hipError_t launch_fp8_linear_direct(const MxMatrix &x, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const MxMatrix &out, hipStream_t stream);

// x, residual, h and y are of one size and type; what is not wanted is nullptr.
struct NormCall {
    MxMatrix x, residual, h, y;
    const void *gain;
    bool gain_fp32;
    double eps;
    int format;
    Fp8Out q;
    float *rstd;
};
hipError_t launch_rms_norm(const NormCall &n, hipStream_t stream);

// Most columns of a backward pass: a row stays in registers.
constexpr int64_t kNormGradCols = 32768;
// Elements of the workspace of a backward pass that sums dgain: a partial row for
// each of its workgroups.  It falls neither with rows nor with cols: what is
// made for the largest pass serves them all.
int64_t norm_grad_partials(int64_t rows, int64_t cols);
struct NormGradCall {
    MxMatrix dy, dh, h, dx;                 // dy: of h's type, or fp32
    const void *gain;
    bool gain_fp32;
    const float *rstd;
    void *dgain;
    float *partial;          // norm_grad_partials(rows, cols) of them
};
hipError_t launch_rms_norm_backward(const NormGradCall &n, hipStream_t stream);

}  // namespace flashopt
