// adamw.cuh -- the AdamW update every optimizer kernel of the library runs.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "shardstate.h"

namespace ss {

// AdamW coefficients, computed once per call on the host in double and
// rounded to fp32.
struct AdamCoef {
    float decay;         // 1 - lr * wd
    float b1, omb1;      // beta1, 1 - beta1
    float b2, omb2;      // beta2, 1 - beta2
    float step_size;     // lr / (1 - beta1^t)
    float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^t)
    float eps;
};

// AdamW update of one element, in fp32.
__device__ __forceinline__ void adamw_elem(float g, float& theta, float& m, float& v,
                                           const AdamCoef& c) {
    theta = __fmul_rn(theta, c.decay);
    m = __fmaf_rn(c.b1, m, __fmul_rn(c.omb1, g));
    v = __fmaf_rn(c.b2, v, __fmul_rn(c.omb2, __fmul_rn(g, g)));
    float denom = __fmaf_rn(__fsqrt_rn(v), c.inv_sqrt_bc2, c.eps);
    theta = __fmaf_rn(-c.step_size, __fdiv_rn(m, denom), theta);
}

inline AdamCoef make_coef(const ss_adamw* hp) {
    AdamCoef c;
    std::memset(&c, 0, sizeof c);
    if (!hp) return c;
    const double t = (double)hp->step;
    const double bc1 = 1.0 - std::pow(hp->beta1, t);
    const double bc2 = 1.0 - std::pow(hp->beta2, t);
    c.decay = (float)(1.0 - hp->lr * hp->weight_decay);
    c.b1 = (float)hp->beta1;
    c.omb1 = (float)(1.0 - hp->beta1);
    c.b2 = (float)hp->beta2;
    c.omb2 = (float)(1.0 - hp->beta2);
    c.step_size = (float)(hp->lr / bc1);
    c.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bc2));
    c.eps = (float)hp->eps;
    return c;
}

// Whether hyper-parameters are ones the update accepts (step t >= 1, betas in
// [0, 1), eps >= 0, finite rate and decay).
inline bool valid_hyper(const ss_adamw* hp) {
    return hp->step >= 1 && hp->beta1 >= 0.0 && hp->beta1 < 1.0 && hp->beta2 >= 0.0 && hp->beta2 < 1.0 &&
           hp->eps >= 0.0 && std::isfinite(hp->lr) && std::isfinite(hp->weight_decay);
}

}  // namespace ss
