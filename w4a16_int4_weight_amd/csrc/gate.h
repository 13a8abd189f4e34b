// The gated block's activations on the device.
#pragma once

#include <hip/hip_runtime.h>

namespace w4a16 {

// a(g) and a'(g) in fp32. kAct: 0 silu g/(1 + e^-g); 1 gelu g Phi(g); 2 gelu's tanh form,
// 0.5 (1 + tanh y) = 1/(1 + e^-2y). The polynomial's argument is clamped at +-30, where
// its logistic is 0 or 1 exactly, so that no infinity meets a zero.
template <int kAct>
__device__ __forceinline__ float gate_prob(float g, float* slope) {
    if constexpr (kAct == 0) {
        const float e = __builtin_amdgcn_rcpf(1.f + __expf(-g));
        *slope = e * (1.f - e);
        return e;
    } else if constexpr (kAct == 1) {
        *slope = 0.3989422804f * __expf(-0.5f * g * g);
        return 0.5f * erfcf(-0.7071067812f * g);
    } else {
        const float y = fminf(fmaxf(g, -30.f), 30.f);
        const float e = __builtin_amdgcn_rcpf(1.f + __expf(-1.5957691216f * y * (1.f + 0.044715f * y * y)));
        *slope = e * (1.f - e) * 1.5957691216f * (1.f + 0.134145f * y * y);
        return e;
    }
}

}  // namespace w4a16
