// Host-side launchers of the sm_100a kernels (internal to libparo).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace paro {

// What a layer's kernel does with its sums (epilogue.cuh): kind kEpiPlain,
// kEpiAct (act, residual) or kEpiGated (act; `out` counts gate and up rows,
// Y has out / 2 columns).
struct Epilogue {
    int kind = 0;
    int act = 0;
    const void* residual = nullptr;   // fp16 [T][out] or null; may be Y
};

struct RotDev {
    int64_t in = 0;         // input features
    int G = 0;              // groups of 128 (tables are built per 128 channels)
    int K = 0;              // rotation layers
    int P = 0;              // active pairs per (layer, 128-channel group)
    int group = 128;        // the layer's group size (64: two groups share each 128-channel table;
                            // 256: G counts 256-channel groups, no Givens tables, mats and rotp64
                            // hold the 256-channel forms)
    uint8_t* rotq = nullptr;       // [K][G] quad exchange blocks (decode prologue)
    float* inv_alpha = nullptr;    // [in] fp32 1/alpha
    uint8_t* rotp64 = nullptr;     // [K][G] blocks of 128 partner bytes + 128 double2 (converter)
    double* alpha64 = nullptr;     // [in] alpha as fp64
    uint8_t* mats = nullptr;       // [G][64 KB] dense per-group rotation (hi, lo fp16; tensor-core operand image)
};

// Bytes of one group's dense rotation image: hi and lo fp16 128 x 128.
constexpr size_t kRotMatBytes = 4 * 128 * 128;
// For 256-channel groups, one image per half of the output channels: hi and
// lo fp16 of 256 (k) x 128 (n).
constexpr size_t kRotMat256Bytes = 4 * 256 * 128;

// Shared memory of an SM (1 KB of it is reserved for each resident CTA), and
// the least that a kernel of this library which allocates tensor memory asks
// for (the single-CTA GEMM with 64 tokens per tile; each of them checks it). A
// kernel that takes a whole SM's tensor memory asks for so much that none of
// them fits beside it.
constexpr size_t kSmSharedBytes = 228 * 1024, kCtaReservedBytes = 1024, kLeastTmemSmem = 58 * 1024;

// 2-D TMA descriptor of a row-major tensor [outer][inner] (driver entry point).
bool encode_tma_2d(CUtensorMap* tm, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

cudaError_t launch_rotate(const RotDev& r, const void* X, void* Xr, int64_t T, cudaStream_t s);
// Tensor-core rotation (dense per-group matrices); any T >= 1.
cudaError_t launch_rotate_tc(const RotDev& r, const void* X, void* Xr, int64_t T, cudaStream_t s);
// X' = X T^-1: Givens kernel up to 16 tokens, tensor-core kernel above.
// Decode batches (1 <= T <= 16): one CTA per group, all layers' parameters in
// shared memory; launched as a programmatic dependent of the previous kernel.
// lane_major: X' is written with every 64-channel block in the decode
// kernel's B-fragment order (channel 16 j + 4 q + e at 16 q + 4 j + e).
cudaError_t launch_rotate_decode(const RotDev& r, const void* X, void* Xr, int64_t T, cudaStream_t s,
                                 bool lane_major = false);
size_t rotate_decode_smem(int K, int T);

// group: channels per quantisation group (128 or 64) of the weight format.
cudaError_t launch_pack(const uint8_t* q, const uint16_t* sc, const uint8_t* z, int64_t in, int64_t out, int group,
                        void* qw, void* scp, void* zp, cudaStream_t s, bool gated = false);
cudaError_t launch_dequant(const void* qw, const void* scp, const void* zp, int64_t in, int64_t out, int group,
                           void* W, cudaStream_t s);
cudaError_t launch_quantize(const RotDev& r, const void* W, int64_t out, uint8_t* q, uint16_t* sc,
                            uint8_t* z, cudaStream_t s);

// Decode path (tokens <= 16): the decode rotation kernel into ws (when rot
// is not null), then the int4 decode kernel, both programmatic dependent launches.
// group: channels per quantisation group of the weights (128 or 64).
// y_fp32: Y is fp32 and receives the unrounded sums (row-parallel partials).
cudaError_t launch_gemv(const RotDev* rot, const void* X, const void* qw, const void* scp, const void* zp,
                        const void* bias, void* Y, int64_t T, int64_t in, int64_t out, int group, void* ws,
                        cudaStream_t s, bool y_fp32 = false, const Epilogue& epi = Epilogue());

// Decode with the X' scratch in a static device array (no allocation anywhere).
size_t noalloc_scratch_bytes();
cudaError_t launch_gemv_noalloc(const RotDev* rot, const void* X, const void* qw, const void* scp, const void* zp,
                                void* Y, int64_t T, int64_t in, int64_t out, cudaStream_t s);

// Prefill (tokens > 16): tcgen05 GEMM on X' (already rotated, in global memory),
// launched as a programmatic dependent of the rotation kernel.
// group: channels per quantisation group of the weights (128 or 64).
cudaError_t launch_gemm(const void* Xr, const void* qw, const void* scp, const void* zp, const void* bias, void* Y,
                        int64_t T, int64_t in, int64_t out, int group, cudaStream_t s, bool y_fp32 = false,
                        const Epilogue& epi = Epilogue());
// Above 16 tokens on CTA pairs (gemm_pair_sm100.cu), with the epilogues kEpiAct and kEpiGated.
cudaError_t launch_gemm_pair(const void* Xr, const void* qw, const void* scp, const void* zp, const void* bias, void* Y,
                             int64_t T, int64_t in, int64_t out, int group, cudaStream_t s, const Epilogue& epi);

// Y16 = fp16(Yf + bias) (bias fp16 [out] or null): the last step of a
// row-parallel layer after the partial sums were added across ranks.
cudaError_t launch_finalize(const float* Yf, const void* bias, void* Y, int64_t T, int64_t out, cudaStream_t s);

// v = x + b + r, H = fp16(v), Y = norm(v) in fp16, or (S not null) e4m3 codes
// with one scale per 128 channels (scale_group != 0) or per row. x fp16 or
// fp32; r, b, H may be null; H may be x or r.
cudaError_t launch_rmsnorm(const void* x, bool x_fp32, const void* r, const void* b, const void* w, float eps, void* H,
                           void* Y, float* S, int scale_group, int64_t T, int64_t F, cudaStream_t s);
// Y = fp16(code * scale)
cudaError_t launch_q8_expand(const void* Q, const float* S, int scale_group, void* Y, int64_t T, int64_t F,
                             cudaStream_t s);

// A kernel whose bounded wait runs out on purpose after limit_ns (fault code 6).
cudaError_t launch_wait_selftest(uint64_t limit_ns, cudaStream_t s);

// Fault code left by a bounded wait that ran out (0 = none); optionally
// cleared. Every source file with bounded waits has a fault word of its own.
cudaError_t read_fault_gemm(unsigned int* code, bool clear);
cudaError_t read_fault_gemm_pair(unsigned int* code, bool clear);
cudaError_t read_fault_rotate(unsigned int* code, bool clear);

}  // namespace paro
