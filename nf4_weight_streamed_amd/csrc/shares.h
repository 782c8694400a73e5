// Sums of the shares that several workgroups leave of one result, in their order.
#pragma once

#include "device.h"

namespace nf4 {

struct Shares {  // dst[i] = ((src[0][i] + src[1][i]) + src[2][i]) + ...
    const float* src;
    int count;
    int64_t total;
    float* dst;
};

__device__ __forceinline__ void sum_shares(const Shares& sh, int64_t block) {
    const int64_t idx = (block * 256 + threadIdx.x) * 4;
    if (idx >= sh.total) return;
    f32x4 a = *reinterpret_cast<const f32x4*>(sh.src + idx);
    for (int z = 1; z < sh.count; ++z) a += *reinterpret_cast<const f32x4*>(sh.src + size_t(z) * sh.total + idx);
    *reinterpret_cast<f32x4*>(sh.dst + idx) = a;
}

}  // namespace nf4
