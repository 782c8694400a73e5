// Activation checkpoints in 8 bits (the format: act8.h), and the SiLU product that keeps its
// inputs in them: what the backward reads, held at 1.0625 bytes an element instead of 2. All
// of it is elementwise within blocks of 64, so rows are taken as one flat array (rows are whole
// blocks): 8 elements a lane, 8 lanes a block, the block's largest by three lane exchanges.
#include "../../include/nf4lora.h"
#include "act8.h"
#include "common.h"

namespace nf4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxElems = int64_t(1) << 34;  // a launch holds 2^32 threads

__device__ __forceinline__ int64_t first_octet() { return int64_t(blockIdx.x) * kThreads + threadIdx.x; }

// Results are stored past the caches: the next operator finds them no later (a training step of four
// 7B layers takes the same time) and this one loses less of its inputs (512 x 18944 SiLU product
// 14.6 -> 13.4 us, its backward 14.3 -> 12.7). Inputs are loaded past them too (kStream) where a call
// moves more than the last-level cache holds: 8192 x 29568 forward 322 -> 313 us, m again 160 -> 146,
// backward 331 -> 312; at 512 rows, whose inputs the previous operator has just written, 13.4 -> 15.0
// and 12.7 -> 15.0. Quantising takes neither (125 us; 127 and 131).
constexpr size_t kLastLevelCache = size_t(256) << 20;

template <bool kStream, typename V>
__device__ __forceinline__ V load(const void* p, int64_t i) {
    const V* q = static_cast<const V*>(p) + i;
    return kStream ? __builtin_nontemporal_load(q) : *q;
}

__device__ __forceinline__ void store_octet(uint16_t* p, int64_t i, const float (&v)[8]) {
    __builtin_nontemporal_store(pack_octet(v), reinterpret_cast<u32x4*>(p) + i);
}

struct Checkpoint {
    const uint8_t* codes;
    const float* scale;
    template <bool kStream>
    __device__ __forceinline__ void read(int64_t i, float (&v)[8]) const {
        act8_values8(load<kStream, u32x2>(codes, i), scale[i >> 3], v);
    }
};

struct CheckpointOut {
    uint8_t* codes;
    float* scale;
    template <bool kPast>
    __device__ __forceinline__ void write(int64_t i, u32x4 x) const {
        float s;
        const u32x2 c = act8_quantize8(x, s);
        u32x2* q = reinterpret_cast<u32x2*>(codes) + i;
        if constexpr (kPast)
            __builtin_nontemporal_store(c, q);
        else
            *q = c;
        if ((i & 7) == 0) scale[i >> 3] = s;
    }
};

__global__ __launch_bounds__(kThreads) void k_act8_quantize(const uint16_t* x, int64_t octets, CheckpointOut out) {
    const int64_t i = first_octet();
    if (i < octets) out.write<false>(i, load<false, u32x4>(x, i));
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void k_act8_dequantize(Checkpoint in, int64_t octets, uint16_t* out) {
    const int64_t i = first_octet();
    if (i >= octets) return;
    float v[8];
    in.read<kStream>(i, v);
    store_octet(out, i, v);
}

// 1 / (1 + e^-z): the hardware's exponential and reciprocal are off by about 2^-22 of the result
// (and by 2^-24 |z| through the exponent's product), far below the bf16 rounding behind them.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void k_silu_mul_fwd_act8(const uint16_t* gate, const uint16_t* up, int64_t octets,
                                                                uint16_t* m, CheckpointOut g8, CheckpointOut u8) {
    const int64_t i = first_octet();
    if (i >= octets) return;
    const u32x4 gw = load<kStream, u32x4>(gate, i), uw = load<kStream, u32x4>(up, i);
    float g[8], u[8];
    unpack_octet(gw, g);
    unpack_octet(uw, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= g[e] * sigmoid(g[e]);
    store_octet(m, i, u);
    g8.write<true>(i, gw);
    u8.write<true>(i, uw);
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void k_silu_mul_act8(Checkpoint g8, Checkpoint u8, int64_t octets, uint16_t* m) {
    const int64_t i = first_octet();
    if (i >= octets) return;
    float g[8], u[8];
    g8.read<kStream>(i, g);
    u8.read<kStream>(i, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= g[e] * sigmoid(g[e]);
    store_octet(m, i, u);
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void k_silu_mul_bwd_act8(Checkpoint g8, Checkpoint u8, const uint16_t* dm, int64_t octets,
                                                                uint16_t* dgate, uint16_t* dup) {
    const int64_t i = first_octet();
    if (i >= octets) return;
    float g[8], u[8], d[8];
    unpack_octet(load<kStream, u32x4>(dm, i), d);
    g8.read<kStream>(i, g);
    u8.read<kStream>(i, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float s = sigmoid(g[e]), t = g[e] * s;
        u[e] *= d[e] * (s + t * (1.0f - s));
        d[e] *= t;
    }
    store_octet(dgate, i, u);
    store_octet(dup, i, d);
}

bool aligned(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

// The arguments of an elementwise call over [rows][cols], checked as they are named. A thread
// reads its elements before it writes them, so an output may be a bf16 input itself.
class Call {
public:
    Call(const char* fn, int64_t rows, int64_t cols) : fn_(fn) {
        if (rows < 0 || cols <= 0 || cols % NF4_BLOCK != 0)
            status_ = fail(NF4_E_SHAPE, "%s: need rows >= 0 and cols a positive multiple of %d (got %lld x %lld)", fn, NF4_BLOCK,
                           (long long)rows, (long long)cols);
        else if (rows > kMaxElems / cols)
            status_ = fail(NF4_E_SHAPE, "%s: at most 2^34 elements (got %lld x %lld)", fn, (long long)rows, (long long)cols);
        else
            elems_ = rows * cols;
    }
    Call& read(const uint16_t* p) { return add(p, 2, false); }
    Call& write(const uint16_t* p) { return add(p, 2, true); }
    Call& read8(const uint8_t* codes, const float* scale) { return add(codes, 1, false).add_scale(scale, false); }
    Call& write8(const uint8_t* codes, const float* scale) { return add(codes, 1, true).add_scale(scale, true); }
    bool nothing() const { return status_ != NF4_OK || elems_ == 0; }
    int status() const { return status_; }
    int64_t octets() const { return elems_ / 8; }
    bool large() const {  // no cache holds what the call moves
        size_t bytes = 0;
        for (int i = 0; i < n_; ++i) bytes += range_[i].bytes;
        return bytes > kLastLevelCache;
    }
    dim3 grid() const { return dim3(unsigned(cdiv(octets(), kThreads))); }

private:
    Call& add(const void* p, int size, bool out) {
        if (nothing()) return *this;
        if (!aligned(p, 16))
            status_ = fail(NF4_E_ARG, "%s: bf16 tensors and codes must be non-NULL and 16-byte aligned", fn_);
        return keep({p, size_t(elems_) * size}, out);
    }
    Call& add_scale(const float* p, bool out) {
        if (nothing()) return *this;
        if (!aligned(p, 4)) status_ = fail(NF4_E_ARG, "%s: scales must be non-NULL and 4-byte aligned", fn_);
        return keep({p, size_t(elems_) / NF4_BLOCK * 4}, out);
    }
    Call& keep(ByteRange r, bool out) {  // inputs are named before outputs
        for (int i = 0; i < n_ && out && status_ == NF4_OK; ++i)
            if (r.meets(range_[i]) && !(i < inputs_ && r.p == range_[i].p && r.bytes == range_[i].bytes))
                status_ = fail(NF4_E_ARG, "%s: an output overlaps another argument (only a bf16 input, exactly, is allowed)", fn_);
        range_[n_++] = r;
        if (!out) inputs_ = n_;
        return *this;
    }
    const char* fn_;
    int status_ = NF4_OK, n_ = 0, inputs_ = 0;
    int64_t elems_ = 0;
    ByteRange range_[8];
};

}  // namespace

}  // namespace nf4

using namespace nf4;

extern "C" {

int nf4_act8_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, float* scale, nf4_stream stream) {
    Call c("nf4_act8_quantize", rows, cols);
    c.read(x).write8(codes, scale);
    if (c.nothing()) return c.status();
    hipLaunchKernelGGL(k_act8_quantize, c.grid(), dim3(kThreads), 0, static_cast<hipStream_t>(stream), x, c.octets(),
                       CheckpointOut{codes, scale});
    return check_launch("nf4_act8_quantize");
}

int nf4_act8_dequantize(const uint8_t* codes, const float* scale, int64_t rows, int64_t cols, uint16_t* x, nf4_stream stream) {
    Call c("nf4_act8_dequantize", rows, cols);
    c.read8(codes, scale).write(x);
    if (c.nothing()) return c.status();
    hipLaunchKernelGGL((c.large() ? k_act8_dequantize<true> : k_act8_dequantize<false>), c.grid(), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), Checkpoint{codes, scale}, c.octets(), x);
    return check_launch("nf4_act8_dequantize");
}

int nf4_silu_mul_fwd_act8(const uint16_t* gate, const uint16_t* up, int64_t rows, int64_t cols, uint16_t* m,
                          uint8_t* gate_codes, float* gate_scale, uint8_t* up_codes, float* up_scale, nf4_stream stream) {
    Call c("nf4_silu_mul_fwd_act8", rows, cols);
    c.read(gate).read(up).write(m).write8(gate_codes, gate_scale).write8(up_codes, up_scale);
    if (c.nothing()) return c.status();
    hipLaunchKernelGGL((c.large() ? k_silu_mul_fwd_act8<true> : k_silu_mul_fwd_act8<false>), c.grid(), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), gate, up, c.octets(), m,
                       CheckpointOut{gate_codes, gate_scale}, CheckpointOut{up_codes, up_scale});
    return check_launch("nf4_silu_mul_fwd_act8");
}

int nf4_silu_mul_act8(const uint8_t* gate_codes, const float* gate_scale, const uint8_t* up_codes, const float* up_scale,
                      int64_t rows, int64_t cols, uint16_t* m, nf4_stream stream) {
    Call c("nf4_silu_mul_act8", rows, cols);
    c.read8(gate_codes, gate_scale).read8(up_codes, up_scale).write(m);
    if (c.nothing()) return c.status();
    hipLaunchKernelGGL((c.large() ? k_silu_mul_act8<true> : k_silu_mul_act8<false>), c.grid(), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), Checkpoint{gate_codes, gate_scale},
                       Checkpoint{up_codes, up_scale}, c.octets(), m);
    return check_launch("nf4_silu_mul_act8");
}

int nf4_silu_mul_bwd_act8(const uint8_t* gate_codes, const float* gate_scale, const uint8_t* up_codes, const float* up_scale,
                          const uint16_t* dm, int64_t rows, int64_t cols, uint16_t* dgate, uint16_t* dup,
                          nf4_stream stream) {
    Call c("nf4_silu_mul_bwd_act8", rows, cols);
    c.read8(gate_codes, gate_scale).read8(up_codes, up_scale).read(dm).write(dgate).write(dup);
    if (c.nothing()) return c.status();
    hipLaunchKernelGGL((c.large() ? k_silu_mul_bwd_act8<true> : k_silu_mul_bwd_act8<false>), c.grid(), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), Checkpoint{gate_codes, gate_scale},
                       Checkpoint{up_codes, up_scale}, dm, c.octets(), dgate, dup);
    return check_launch("nf4_silu_mul_bwd_act8");
}

}  // extern "C"
