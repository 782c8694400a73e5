// Rotary positions on q and k, with several position axes (time, height, width for images
// and video; one axis is the text decoder's). Pair i of a head is its elements i and
// i + D/2; it belongs to one axis x(i) and is turned by phi = pos[x(i)][t] * inv_freq[i]:
//   lo' = lo cos phi - hi sin phi,   hi' = hi cos phi + lo sin phi
// (the inverse, which is the gradient's direction, by -phi). Rotating is elementwise, so
// the bound is reading and writing q and k once. The angle is formed in fp64 and reduced to
// a fraction of a turn before it is rounded to fp32: at position 10^6 an fp32 product would
// be off by 0.06 radians. A token's D/2 cosines and sines are formed once per workgroup
// (one thread each) and shared by all its heads through LDS. 8192 tokens of 64/8 heads of 128
// (302 MB read and written): 50 us, 6.0 TB/s; one token of 28/4 heads: 1.9 us, a launch.
#include "../../include/nf4lora.h"
#include "common.h"
#include "device.h"

namespace nf4 {

namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    const int32_t* pos;      // [axes][T]
    const double* inv_freq;  // [D/2]
    int64_t T;
    int hq, hkv, D, tokens;  // tokens of a workgroup
    int axis_end[4];         // pairs below axis_end[x] (and not below an earlier end) take axis x
    float sign;
};

__global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a) {
    __shared__ __align__(16) float sCos[kThreads], sSin[kThreads];  // [token][pair]
    const int half = a.D / 2, tid = threadIdx.x;
    const int64_t t0 = int64_t(blockIdx.x) * a.tokens;
    const int nt = int(min(int64_t(a.tokens), a.T - t0));
    if (tid < nt * half) {
        const int i = tid % half;
        int axis = 0;
        while (axis < 3 && i >= a.axis_end[axis]) ++axis;
        constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double turns = double(a.pos[axis * a.T + t0 + tid / half]) * (a.inv_freq[i] * kTurn);
        float s, c;
        sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
        sCos[tid] = c;
        sSin[tid] = a.sign * s;
    }
    __syncthreads();
    const int octets = half / 8, heads = a.hq + a.hkv, items = nt * heads * octets;
    for (int n = tid; n < items; n += kThreads) {
        const int oc = n % octets, th = n / octets, head = th % heads, tok = th / heads;
        const bool is_k = head >= a.hq;
        const int64_t row = (t0 + tok) * (is_k ? a.hkv : a.hq) + (is_k ? head - a.hq : head);
        const size_t at = size_t(row) * a.D + 8 * oc;
        const uint16_t* src = (is_k ? a.k : a.q) + at;
        uint16_t* dst = (is_k ? a.k_out : a.q_out) + at;
        const u32x4 lo = *reinterpret_cast<const u32x4*>(src), hi = *reinterpret_cast<const u32x4*>(src + half);
        const float* c = sCos + tok * half + 8 * oc;
        const float* s = sSin + tok * half + 8 * oc;
        u32x4 lo2, hi2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float l0 = __uint_as_float(lo[e] << 16), l1 = __uint_as_float(lo[e] & 0xFFFF0000u);
            const float h0 = __uint_as_float(hi[e] << 16), h1 = __uint_as_float(hi[e] & 0xFFFF0000u);
            lo2[e] = pack_bf16x2(l0 * c[2 * e] - h0 * s[2 * e], l1 * c[2 * e + 1] - h1 * s[2 * e + 1]);
            hi2[e] = pack_bf16x2(h0 * c[2 * e] + l0 * s[2 * e], h1 * c[2 * e + 1] + l1 * s[2 * e + 1]);
        }
        *reinterpret_cast<u32x4*>(dst) = lo2;
        *reinterpret_cast<u32x4*>(dst + half) = hi2;
    }
}

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

}  // namespace

}  // namespace nf4

using namespace nf4;

extern "C" int nf4_rope(const uint16_t* q, const uint16_t* k, int64_t T, int64_t hq, int64_t hkv, int64_t head_dim,
                        const int32_t* pos, const double* inv_freq, const int* sections, int n_axes, int inverse,
                        uint16_t* q_out, uint16_t* k_out, nf4_stream stream) {
    const char* fn = "nf4_rope";
    if (T < 0 || T > (int64_t(1) << 23) || hq < 0 || hkv < 0 || hq > 1024 || hkv > 1024)
        return fail(NF4_E_SHAPE, "%s: need 0 <= T <= 2^23, 0 <= hq, hkv <= 1024 (got T=%lld hq=%lld hkv=%lld)", fn,
                    (long long)T, (long long)hq, (long long)hkv);
    if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0)
        return fail(NF4_E_SHAPE, "%s: head_dim must be a multiple of 16 up to 256 (got %lld)", fn, (long long)head_dim);
    if (n_axes < 1 || n_axes > 4 || !sections)
        return fail(NF4_E_ARG, "%s: need sections for 1 to 4 axes (got n_axes=%d)", fn, n_axes);
    if (inverse != 0 && inverse != 1) return fail(NF4_E_ARG, "%s: inverse must be 0 or 1 (got %d)", fn, inverse);
    RopeArgs a{};
    int64_t sum = 0;
    for (int x = 0; x < n_axes; ++x) {
        if (sections[x] < 1 || sections[x] > 128)
            return fail(NF4_E_ARG, "%s: section %d has %d pairs", fn, x, sections[x]);
        sum += sections[x];
        a.axis_end[x] = int(sum);
    }
    for (int x = n_axes; x < 4; ++x) a.axis_end[x] = int(sum);
    if (sum != head_dim / 2)
        return fail(NF4_E_ARG, "%s: the sections hold %lld pairs, head_dim/2 = %lld", fn, (long long)sum,
                    (long long)(head_dim / 2));
    if (T == 0 || hq + hkv == 0) return NF4_OK;
    if ((hq && (!aligned16(q) || !aligned16(q_out))) || (hkv && (!aligned16(k) || !aligned16(k_out))))
        return fail(NF4_E_ARG, "%s: q, k and the outputs must be non-NULL and 16-byte aligned", fn);
    if (!pos || reinterpret_cast<uintptr_t>(pos) % 4 != 0 || !inv_freq || reinterpret_cast<uintptr_t>(inv_freq) % 8 != 0)
        return fail(NF4_E_ARG, "%s: pos must be 4-byte and inv_freq 8-byte aligned and non-NULL", fn);
    const size_t q_bytes = size_t(T) * hq * head_dim * 2, k_bytes = size_t(T) * hkv * head_dim * 2;
    const ByteRange rq{q, q_bytes}, rk{k, k_bytes}, wq{q_out, q_bytes}, wk{k_out, k_bytes};
    const ByteRange rp{pos, size_t(T) * n_axes * 4}, rf{inv_freq, size_t(head_dim) * 4};
    if (wq.meets(wk) || wq.meets(rk) || wk.meets(rq) || wq.meets(rp) || wq.meets(rf) || wk.meets(rp) || wk.meets(rf) ||
        (q != q_out && wq.meets(rq)) || (k != k_out && wk.meets(rk)))
        return fail(NF4_E_ARG, "%s: an output overlaps another argument (only its own input, exactly, is allowed)", fn);
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out, a.pos = pos, a.inv_freq = inv_freq, a.T = T;
    a.hq = int(hq), a.hkv = int(hkv), a.D = int(head_dim), a.sign = inverse ? -1.0f : 1.0f;
    a.tokens = kThreads / (a.D / 2);
    hipLaunchKernelGGL(k_rope, dim3(unsigned(cdiv(T, a.tokens))), dim3(kThreads), 0, static_cast<hipStream_t>(stream), a);
    return check_launch(fn);
}
