// Sums of the shares that several workgroups leave of one result, in their order.
#pragma once

#include "device.h"

namespace nf4 {

// ((p[0] + p[stride]) + p[2 stride]) + ..., four neighbours at a time. One load a turn would leave a thread waiting for
// each: eight are under way (past the last share, the last again, unused).
__device__ __forceinline__ f32x4 sum_slots(const float* p, int count, size_t stride) {
    constexpr int kAtOnce = 8;
    f32x4 a = *reinterpret_cast<const f32x4*>(p);
    for (int z = 1; z < count; z += kAtOnce) {
        f32x4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) v[i] = *reinterpret_cast<const f32x4*>(p + size_t(min(z + i, count - 1)) * stride);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (z + i < count) a += v[i];
    }
    return a;
}

struct Shares {  // dst[i] = ((src[0][i] + src[1][i]) + src[2][i]) + ...
    const float* src;
    int count;
    int64_t total;
    float* dst;
};

__device__ __forceinline__ void sum_shares(const Shares& sh, int64_t block) {
    const int64_t idx = (block * 256 + threadIdx.x) * 4;
    if (idx >= sh.total) return;
    *reinterpret_cast<f32x4*>(sh.dst + idx) = sum_slots(sh.src + idx, sh.count, size_t(sh.total));
}

}  // namespace nf4
