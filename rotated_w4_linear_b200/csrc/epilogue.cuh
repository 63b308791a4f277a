// What the layer's kernels do with a finished fp32 sum before its rounding to
// fp16: the activations, and the three epilogues the kernels are built with.
#pragma once

#include <math.h>

namespace paro {

// Y = sum + b;  Y = act(sum + b) + residual;  H = act(gate + b_g) (up + b_u),
// gate and up rows interleaved in eights (rows g and g + 8 of a 16-row block)
enum : int { kEpiPlain = 0, kEpiAct = 1, kEpiGated = 2 };

enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4, kActCount = 5 };

// x / (1 + e^-z): the fast exponential and quotient are good to about 2^-20
// here, far below the fp16 rounding of the result; e^-z = inf gives 0 as it should.
__device__ __forceinline__ float gate_by_sigmoid(float x, float z) { return __fdividef(x, 1.f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_fn(float v) {
    if (ACT == kActRelu) return v < 0.f ? 0.f : v;                    // a NaN stays a NaN
    if (ACT == kActSilu) return gate_by_sigmoid(v, v);
    // v Phi(v) with the complementary error function: exact to its relative
    // error in the negative tail, where 1 + erf cancels
    if (ACT == kActGelu) return 0.5f * v * erfcf(-0.70710678118654752f * v);
    // v/2 (1 + tanh u) = v / (1 + e^-2u), u = sqrt(2/pi) (v + 0.044715 v^3)
    if (ACT == kActGeluTanh) return gate_by_sigmoid(v, 1.5957691216057308f * fmaf(0.044715f * v * v, v, v));
    return v;
}

__device__ __forceinline__ float act_any(float v, int act) {          // few elements per thread
    switch (act) {
        case kActRelu: return act_fn<kActRelu>(v);
        case kActSilu: return act_fn<kActSilu>(v);
        case kActGelu: return act_fn<kActGelu>(v);
        case kActGeluTanh: return act_fn<kActGeluTanh>(v);
        default: return v;
    }
}

// fn.template operator()<ACT>() for the runtime activation: the switch stands
// outside the loops over elements.
template <class F>
__device__ __forceinline__ void with_act(int act, const F& fn) {
    switch (act) {
        case kActRelu: fn.template run<kActRelu>(); break;
        case kActSilu: fn.template run<kActSilu>(); break;
        case kActGelu: fn.template run<kActGelu>(); break;
        case kActGeluTanh: fn.template run<kActGeluTanh>(); break;
        default: fn.template run<kActNone>(); break;
    }
}

}  // namespace paro
