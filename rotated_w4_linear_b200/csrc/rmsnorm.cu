// Root-mean-square norm between the layers, with the residual's addition:
//
//   v = x + b + r               (fp32; b and r optional)
//   H = fp16(v)                 (the new residual stream)
//   y = (v w) / sqrt(mean(v^2) + eps)
//   Y = fp16(y), or the codes e4m3(y / s) with s = max|y| / 448 over 128
//       channels or over the row
//
// x is fp16 (a layer's output) or fp32 (the summed shares of a row-parallel
// layer: this kernel then also does the bias and the rounding that
// paro_finalize does on its own). The norm is taken of the unrounded fp32 v,
// so Y carries one rounding only.
//
// Bound: HBM, one pass. A row stays in registers from its loads to its
// stores (VPT vectors of 8 channels per thread), so x and r are read once and
// H and Y written once; the row's sum of squares and its largest |v w| (the
// row's scale: max|y| = max|v w| / rms exactly, since one rounded product is
// monotonic) share one cross-warp reduction in a fixed order, so a row's
// result does not depend on the batch. A 128-channel group is sixteen
// neighbouring lanes, so its largest |v w| is a four-step shuffle, done before
// the row's barrier too.
// Measured (fp16 x, residual and H; HBM copy peak 6552 GB/s): 8192 x 4096
// 42.0-43.0 us, 6250-6390 GB/s; 4096 x 5120 with codes 25.9 us (128 channels
// per scale) and 28.0 us (one scale per row), 5660 and 5250 GB/s; 2048 x 8192
// from fp32 27.1 us, 6190 GB/s; one token of 4096 1.5 us, which is launch and
// latency. A persistent form with a three-deep cp.async ring of rows ran
// slower (50.2 and 30.0 us): enough CTAs are resident that one's loads cover
// another's reduction.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace paro {

namespace {

constexpr float kE4m3Max = 448.f;
// smallest scale: keeps 1/s finite; an all-zero group has this scale and zero codes
constexpr float kScaleFloor = 7.888609052210118e-31f;      // 2^-100

struct NormArgs {
    const void* x;               // fp16 or fp32 [T][F]
    const __half* r;             // fp16 [T][F] or null
    const __half* b;             // fp16 [F] or null
    const __half* w;             // fp16 [F]
    __half* H;                   // fp16 [T][F] or null (may be x or r)
    void* Y;                     // fp16 or e4m3 [T][F]
    float* S;                    // fp32 [T][nscale] (8-bit output)
    int64_t T;
    int nvec;                    // F / 8
    int wpr;                     // warps per row
    int rows;                    // rows per tile
    float inv_f, eps;            // 1 / F
};

__device__ __forceinline__ void unpack8(const uint4& u, float f[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
// f += the eight halves, each sum rounded once to fp32: in one instruction
// per channel (MIXED) or, with the same result, a conversion and a sum.
template <bool MIXED>
__device__ __forceinline__ void add8(float f[8], const uint4& u) {
    if (MIXED) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.f16 %0, lo, %0;\n\t"
                "add.rn.f32.f16 %1, hi, %1;\n\t}"
                : "+f"(f[2 * i]), "+f"(f[2 * i + 1]) : "r"(w[i]));
    } else {
        float t[8];
        unpack8(u, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += t[e];
    }
}
__device__ __forceinline__ uint4 pack8(const float f[8]) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {   // a in the lowest byte
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The scale of channels whose largest |v w| is m, and k = rms / scale, so that
// a code takes one product: e4m3(v w k). The approximate quotient is off by
// 2^-22, the codes' own rounding by up to 2^-4.
__device__ __forceinline__ float q8_scale(float m, float rms, float& k) {
    const float s = fmaxf(m * rms * (1.f / kE4m3Max), kScaleFloor);
    k = __fdividef(rms, s);
    return s;
}
// The warp's largest of values without a sign: their bits compare as integers
// do (a NaN comes out on top; its row's scale is then the floor).
__device__ __forceinline__ float warp_max(float v) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

}  // namespace

enum : int { kNormF16 = 0, kNormQ8Group = 1, kNormQ8Row = 2 };

namespace {

// A thread's place: warps wr of row rw of the CTA's tile of rows.
struct NormPlace {
    int lane, warp, rw, wr, t0, tr;
};
__device__ __forceinline__ NormPlace norm_place(const NormArgs& a) {
    NormPlace p;
    p.lane = threadIdx.x & 31;
    p.warp = threadIdx.x >> 5;
    p.rw = a.rows == 1 ? 0 : p.warp / a.wpr;               // (a division costs as much as a vector's arithmetic)
    p.wr = p.warp - p.rw * a.wpr;
    p.t0 = p.wr * 32 + p.lane;                             // first vector of the row, then every tr-th
    p.tr = a.wpr * 32;
    return p;
}

// The widest rows fetch the weights, which all rows share, when they need
// them: 64 registers a thread do not hold them too.
template <int VPT>
struct NormWeights {
    static constexpr bool kHold = VPT <= 2;
    uint4 w[kHold ? VPT : 1];
    __device__ __forceinline__ void load(const NormArgs& a, const NormPlace& p) {
        if (kHold)
#pragma unroll
            for (int j = 0; j < VPT; ++j) w[j] = fetch(a, p.t0 + j * p.tr);
    }
    __device__ __forceinline__ uint4 get(const NormArgs& a, int j, int i) { return kHold ? w[j] : fetch(a, i); }
    static __device__ __forceinline__ uint4 fetch(const NormArgs& a, int i) {
        return i < a.nvec ? __ldg(reinterpret_cast<const uint4*>(a.w) + i) : make_uint4(0, 0, 0, 0);
    }
};

// Everything after the loads, for one row: v[j] holds x of vector t0 + j tr
// on entry (zeros outside the row), r its residual. Every thread of the CTA
// calls it (it has a barrier).
template <int VPT, int OUT, bool MIXED>
__device__ __forceinline__ void norm_row(const NormArgs& a, const NormPlace& p, int64_t row, bool live,
                                         float (&v)[VPT][8], const uint4 (&r)[VPT], NormWeights<VPT>& w,
                                         float2* part) {
    float ss = 0.f, mx = 0.f;
    float gm[VPT];                                         // largest |v w| of the vector's 128 channels
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = p.t0 + j * p.tr;
        float f[8];
        if (a.b && i < a.nvec) add8<MIXED>(v[j], __ldg(reinterpret_cast<const uint4*>(a.b) + i));
        add8<MIXED>(v[j], r[j]);
        if (a.H && live && i < a.nvec) reinterpret_cast<uint4*>(a.H)[row * a.nvec + i] = pack8(v[j]);
        unpack8(w.get(a, j, i), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(v[j][e], v[j][e], ss);
            v[j][e] *= f[e];                               // v w from here on
        }
        if (OUT != kNormF16) {
            gm[j] = fabsf(v[j][0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) gm[j] = fmaxf(gm[j], fabsf(v[j][e]));
            mx = fmaxf(mx, gm[j]);
        }
        if (OUT == kNormQ8Group)                           // lanes 0-15 and 16-31 are one group each
#pragma unroll
            for (int o = 8; o; o >>= 1) gm[j] = fmaxf(gm[j], __shfl_xor_sync(0xffffffffu, gm[j], o));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (OUT == kNormQ8Row) mx = warp_max(mx);
    if (a.wpr > 1) {
        if (p.lane == 0) part[p.warp] = make_float2(ss, mx);
        __syncthreads();
        const float2 q = p.lane < a.wpr ? part[p.rw * a.wpr + p.lane] : make_float2(0.f, 0.f);
        ss = q.x;
        mx = q.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        if (OUT == kNormQ8Row) mx = warp_max(mx);
    }
    float rms = rsqrtf(ss * a.inv_f + a.eps);        // 2 ulp; infinity gives 0
    if (OUT != kNormF16 && rms > 1.34217728e8f) {          // 2^27: k could overflow, so v w takes rms at once
        mx *= rms;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            gm[j] *= rms;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] *= rms;
        }
        rms = 1.f;
    }
    float k = rms;                                         // v w k: the norm, or the norm over its scale
    if (OUT == kNormQ8Row) {
        const float s = q8_scale(mx, rms, k);
        if (live && p.wr == 0 && p.lane == 0) a.S[row] = s;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = p.t0 + j * p.tr;
        const bool in = live && i < a.nvec;
        if (OUT == kNormQ8Group) {
            const float s = q8_scale(gm[j], rms, k);
            if (in && (p.lane & 15) == 0) a.S[row * ((a.nvec + 15) >> 4) + (i >> 4)] = s;
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[j][e] * k;
        if (!in) continue;
        if (OUT == kNormF16)
            static_cast<uint4*>(a.Y)[row * a.nvec + i] = pack8(y);
        else
            static_cast<uint2*>(a.Y)[row * a.nvec + i] =
                make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
    }
}

template <bool X32>
__device__ __forceinline__ void unpack_x(const uint4 (&x)[X32 ? 2 : 1], float v[8]) {
    if (X32) {
#pragma unroll
        for (int h = 0; h < (X32 ? 2 : 1); ++h) {
            v[4 * h] = __uint_as_float(x[h].x);
            v[4 * h + 1] = __uint_as_float(x[h].y);
            v[4 * h + 2] = __uint_as_float(x[h].z);
            v[4 * h + 3] = __uint_as_float(x[h].w);
        }
    } else {
        unpack8(x[0], v);
    }
}

}  // namespace

// REGS, registers per thread, are held to what keeps as many warps resident
// as the loads need: an SM quarter holds 16 warps at 32, 12 at 40, 10 at 48,
// 8 at 64 and 7 at 72 (see launch_rmsnorm).
template <int VPT, bool X32, int OUT, int REGS>
__global__ void __maxnreg__(REGS) rmsnorm_kernel(const NormArgs a) {
    // the next kernel may launch; it reads nothing of ours before this grid is complete
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int XV = X32 ? 2 : 1;
    __shared__ float2 part[32];                            // per warp: sum of squares, largest |v w|
    const NormPlace p = norm_place(a);
    const int64_t row = (int64_t)blockIdx.x * a.rows + p.rw;
    const bool live = row < a.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");     // x and r may be the previous grid's output
    // every load of the row in flight before any is used
    uint4 x[VPT][XV], r[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = p.t0 + j * p.tr;
        const bool in = live && i < a.nvec;
        const int64_t at = row * a.nvec + i;
#pragma unroll
        for (int h = 0; h < XV; ++h) {
            x[j][h] = make_uint4(0, 0, 0, 0);
            if (in) x[j][h] = static_cast<const uint4*>(a.x)[at * XV + h];
        }
        r[j] = make_uint4(0, 0, 0, 0);
        if (in && a.r) r[j] = reinterpret_cast<const uint4*>(a.r)[at];
    }
    NormWeights<VPT> w;
    w.load(a, p);
    float v[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) unpack_x<X32>(x[j], v[j]);
    // Mixed sums pay where x is fp32 and the codes have a scale per 128 channels
    // (4882 x 5120: 35.5 us against 38.2, 3051 x 8192: 36.8 against 41.0); the
    // other forms gain nothing or lose to the order that the compiler then
    // gives their loads (4882 x 5120, fp16 throughout: 33.9 against 31.9).
    norm_row<VPT, OUT, X32 && OUT == kNormQ8Group && VPT <= 2>(a, p, row, live, v, r, w, part);
}

// Codes and scales back to fp16: Y = fp16(code s). Eight channels per thread;
// bound by HBM (3 bytes per channel).
__global__ void q8_expand_kernel(const uint2* __restrict__ Q, const float* __restrict__ S, uint4* __restrict__ Y,
                                 int nvec, int nscale, int64_t n) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (k >= n) return;
    const int64_t row = k / nvec;
    const int i = (int)(k - row * nvec);
    const uint2 q = Q[k];
    const float s = S[row * nscale + (nscale > 1 ? i >> 4 : 0)];
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {                          // two codes -> two fp16 (exact), then one rounded product
        const uint16_t c = (uint16_t)((e < 2 ? q.x : q.y) >> (16 * (e & 1)));
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        y[2 * e] = f.x * s;
        y[2 * e + 1] = f.y * s;
    }
    Y[k] = pack8(y);
}

namespace {

cudaLaunchConfig_t pdl_config(unsigned grid, unsigned block, cudaStream_t s, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int VPT, bool X32, int OUT, int REGS>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        pdl_config((unsigned)((a.T + a.rows - 1) / a.rows), (unsigned)(32 * a.wpr * a.rows), s, &attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rmsnorm_kernel<VPT, X32, OUT, REGS>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int VPT, bool X32, int REGS>
cudaError_t launch_norm_out(const NormArgs& a, int out, cudaStream_t s) {
    return out == kNormF16       ? launch_norm<VPT, X32, kNormF16, REGS>(a, s)
           : out == kNormQ8Group ? launch_norm<VPT, X32, kNormQ8Group, REGS>(a, s)
                                 : launch_norm<VPT, X32, kNormQ8Row, REGS>(a, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, bool x_fp32, const void* r, const void* b, const void* w, float eps, void* H,
                           void* Y, float* S, int scale_group, int64_t T, int64_t F, cudaStream_t s) {
    if (T <= 0) return cudaSuccess;
    NormArgs a{};
    a.x = x;
    a.r = static_cast<const __half*>(r);
    a.b = static_cast<const __half*>(b);
    a.w = static_cast<const __half*>(w);
    a.H = static_cast<__half*>(H);
    a.Y = Y;
    a.S = S;
    a.T = T;
    a.nvec = (int)(F / 8);
    a.inv_f = (float)(1.0 / (double)F);
    a.eps = eps;
    const int out = !S ? kNormF16 : scale_group ? kNormQ8Group : kNormQ8Row;
    // The split of a row over threads goes by its width (and the type of x)
    // alone, so a row's sums have the same order in every batch: one vector
    // per thread up to 11 warps, then two, then four where two would leave
    // one CTA on an SM (above 20 warps at 48 registers). Measured: 8192 x 4096
    // 42.0 us with two, 43.0 with one; 8192 x 2560 from fp32 32.8 with one,
    // 34.1 with two; 2034 x 12288 34.1 with four, 40.9 with two, and with a
    // scale per row 35.5 against 44.4; from fp32 42.3 against 44.4. Four
    // vectors of fp32 take 72 registers (with 64, which spill, 45.7), which leave
    // one CTA above 14 warps: there two vectors again while they fit (1525 x
    // 16384 from fp32 43.0, with four 49.1).
    const int nw = (a.nvec + 31) / 32;                      // warps at one vector per thread
    const int vpt = nw <= 11 ? 1 : nw <= 40 || (x_fp32 && nw > 56 && nw <= 64) ? 2 : 4;
    a.wpr = (nw + vpt - 1) / vpt;
    a.rows = T > 296 && a.wpr < 8 ? 8 / a.wpr : 1;
    if (x_fp32) {
        if (vpt == 1) return launch_norm_out<1, true, 32>(a, out, s);
        if (vpt == 2) return launch_norm_out<2, true, 48>(a, out, s);
        return a.wpr <= 28 ? launch_norm_out<4, true, 72>(a, out, s)
                           : launch_norm_out<4, true, 64>(a, out, s);   // 32 warps fit
    }
    if (vpt == 1) return launch_norm_out<1, false, 32>(a, out, s);
    if (vpt == 4) return launch_norm_out<4, false, 64>(a, out, s);
    // A scale per row has the longest way from its loads to its stores: where
    // 40 registers (4 bytes spilled) let one more CTA in than 48, it gains
    // (3051 x 8192 32.0 us against 36.2; where they do not, 5120 wide, 33.4
    // against 32.8). The other outputs do not: 6144 wide 33.4 against 32.1.
    if (out == kNormQ8Row && 48 / a.wpr > 40 / a.wpr) return launch_norm<2, false, kNormQ8Row, 40>(a, s);
    return launch_norm_out<2, false, 48>(a, out, s);
}

cudaError_t launch_q8_expand(const void* Q, const float* S, int scale_group, void* Y, int64_t T, int64_t F,
                             cudaStream_t s) {
    if (T <= 0) return cudaSuccess;
    const int nvec = (int)(F / 8);
    const int64_t n = T * nvec;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((unsigned)((n + 255) / 256), 256u, s, &attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, q8_expand_kernel, static_cast<const uint2*>(Q), S,
                                             static_cast<uint4*>(Y), nvec,
                                             scale_group ? (int)((F + 127) / 128) : 1, n);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paro
