// The residual stream around a block: the block's output o, normalised and gated, joins the
// stream h, and the next block's input is the stream normalised. Per row of H elements:
//   v = o  or  o rstd_o (off + post_gain),   rstd_o = 1 / sqrt(mean o^2 + eps)
//   s = h + scale gate v,   h' = RNbf(s),   rstd = 1 / sqrt(mean s^2 + eps)
//   n = RNbf(s rstd (off + gain)),   and n's 8-bit checkpoint (act8.h)
// and back, with g the sum of the gradients of n's readers, b = h' rstd or the checkpoint's
// value, w = g (off + gain), u = o rstd_o (or o):
//   ds = dres + rstd (w - b mean(w b)),   dh = RNbf(ds),   dgain = sum_t g b
//   dv = scale ds,   dgate = dv v,   then dv <- dv gate
//   dpost_gain = sum_t dv u,   p = dv (off + post_gain),   do = rstd_o (p - u mean(p u))  or  dv
// A row is held in registers between its reductions, so that every tensor is read once and
// written once; that traffic is the bound. All arithmetic is fp32. Sums over rows (gains, a
// gate a channel) are kept per column in registers over a workgroup's rows, then added over
// the workgroups by a second kernel, in a fixed order.
#include <cmath>

#include "../../include/nf4lora.h"
#include "act8.h"
#include "common.h"

namespace nf4 {

namespace {

constexpr int64_t kMaxWidth = 16384;
constexpr int64_t kMaxGrid = int64_t(1) << 21;  // workgroups; rows past it are looped over

// Eight elements of a row from column `at` on; zeros past its end. kRagged: rows that are no
// whole number of 16-byte pieces, or not aligned to them.
struct __attribute__((packed, aligned(2))) LooseOctet {
    u32x4 w;
};

template <bool kRagged>
__device__ __forceinline__ u32x4 load_octet(const uint16_t* row, int at, int H) {
    if constexpr (!kRagged) return at < H ? *reinterpret_cast<const u32x4*>(row + at) : u32x4{0, 0, 0, 0};
    if (at + 8 <= H) return reinterpret_cast<const LooseOctet*>(row + at)->w;
    u32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (at + e < H) x[e / 2] |= uint32_t(row[at + e]) << (16 * (e % 2));
    return x;
}

template <bool kRagged>
__device__ __forceinline__ void store_octet(uint16_t* row, int at, int H, u32x4 x) {
    if constexpr (!kRagged) {
        if (at < H) *reinterpret_cast<u32x4*>(row + at) = x;
        return;
    }
    if (at + 8 <= H) {
        reinterpret_cast<LooseOctet*>(row + at)->w = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (at + e < H) row[at + e] = uint16_t(x[e / 2] >> (16 * (e % 2)));
}

__device__ __forceinline__ float lane_sum(float v) {
    auto other = [](float w, auto c) {
        return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(w), __float_as_int(w), decltype(c)::value, 0xF, 0xF, false));
    };
    v += other(v, std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
    v += other(v, std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
    v += other(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
    v += other(v, std::integral_constant<int, 0x140>{});  // row_mirror
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// Sum over the TR threads of a row, in a fixed order. Two slots taken in turn need one barrier
// a sum: whoever writes a slot again has met the barrier that followed its last reads.
template <int TR>
struct RowSum {
    float (&slots)[2][16];
    int turn = 0;
    __device__ __forceinline__ float operator()(float v) {
        v = lane_sum(v);
        if constexpr (TR == 64) return v;
        float(&slot)[16] = slots[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        float s = slot[0];
#pragma unroll
        for (int i = 1; i < TR / 64; ++i) s += slot[i];
        return s;
    }
};

// TR threads a row, N octets a thread: octet n of thread t starts at column 8 (n TR + t).
template <int TR>
constexpr int kRowsOf = TR < 256 ? 256 / TR : 1;  // rows of a workgroup
template <int TR>
constexpr int kBlock = TR < 256 ? 256 : TR;

struct FwdArgs {
    const uint16_t *h, *o, *post_gain, *gate, *gain;
    uint16_t *h_out, *n;
    uint8_t* codes;
    float *n_scale, *rstd_o, *rstd;
    int64_t T;
    int H, post, gate_kind;
    float scale, offset, eps;
};

// factor of column at + e: 1 without a gain
template <bool kRagged>
__device__ __forceinline__ void gain_octet(const uint16_t* gain, float offset, int at, int H, float (&f)[8]) {
    if (!gain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 1.0f;
        return;
    }
    unpack_octet(load_octet<kRagged>(gain, at, H), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += offset;
}

template <int TR, int N, bool kRagged>
__global__ __launch_bounds__(kBlock<TR>) void k_residual_norm_fwd(FwdArgs a) {
    constexpr int R = kRowsOf<TR>;
    __shared__ float slots[2][16];
    RowSum<TR> row_sum{slots};
    const int t = threadIdx.x % TR, H = a.H;
    const float mean = 1.0f / float(H);
    for (int64_t row = int64_t(blockIdx.x) * R + threadIdx.x / TR; row < a.T; row += int64_t(gridDim.x) * R) {
        const int64_t base = row * H;
        u32x4 hw[N], ow[N], gw[N];
#pragma unroll
        for (int n = 0; n < N; ++n) hw[n] = load_octet<kRagged>(a.h + base, 8 * (n * TR + t), H);
        if (a.o) {
#pragma unroll
            for (int n = 0; n < N; ++n) ow[n] = load_octet<kRagged>(a.o + base, 8 * (n * TR + t), H);
            if (a.gate_kind != NF4_GATE_NONE) {
                const uint16_t* g = a.gate + (a.gate_kind == NF4_GATE_TOKEN ? base : 0);
#pragma unroll
                for (int n = 0; n < N; ++n) gw[n] = load_octet<kRagged>(g, 8 * (n * TR + t), H);
            }
        }
        float s[N][8];
#pragma unroll
        for (int n = 0; n < N; ++n) unpack_octet(hw[n], s[n]);
        if (a.o) {
            float r = 1.0f;
            if (a.post) {
                float ss = 0.0f;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float v[8];
                    unpack_octet(ow[n], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
                }
                r = 1.0f / sqrtf(row_sum(ss) * mean + a.eps);
                if (t == 0) a.rstd_o[row] = r;
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at = 8 * (n * TR + t);
                float v[8], f[8];
                unpack_octet(ow[n], v);
                if (a.post) {
                    gain_octet<kRagged>(a.post_gain, a.offset, at, H, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = v[e] * r * f[e];
                }
                if (a.gate_kind != NF4_GATE_NONE) {
                    unpack_octet(gw[n], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= f[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s[n][e] = __builtin_fmaf(a.scale, v[e], s[n][e]);
                store_octet<kRagged>(a.h_out + base, at, H, pack_octet(s[n]));
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(s[n][e], s[n][e], ss);
        const float r = 1.0f / sqrtf(row_sum(ss) * mean + a.eps);
        if (t == 0) a.rstd[row] = r;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = 8 * (n * TR + t);
            float f[8];
            gain_octet<kRagged>(a.gain, a.offset, at, H, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s[n][e] * r;
            const u32x4 w = pack_octet(f);
            store_octet<kRagged>(a.n + base, at, H, w);
            if (a.codes && at < H) {  // H % 64 == 0: the 8 lanes of a block are all in or all out
                float step;
                *reinterpret_cast<u32x2*>(a.codes + base + at) = act8_quantize8(w, step);
                if ((t & 7) == 0) a.n_scale[(base + at) >> 6] = step;
            }
        }
    }
}

struct BwdArgs {
    const uint16_t *dn[3], *dres, *h, *o, *post_gain, *gate, *gain;
    const uint8_t* codes;
    const float *n_scale, *rstd, *rstd_o;
    uint16_t *dh, *d_o, *dgate_rows;
    float* part;  // [workgroups][dgain, dpost_gain, dgate][H]; which are wanted:
    int sums;     // bit 0, 1, 2
    int64_t T;
    int H, n_dn, post, gate_kind;
    float scale, offset;
};

// kSums: sums over rows are wanted; a workgroup then takes every gridDim-th row.
template <int TR, int N, bool kRagged, bool kSums>
__global__ __launch_bounds__(kBlock<TR>) void k_residual_norm_bwd(BwdArgs a) {
    constexpr int R = kRowsOf<TR>;
    static_assert(!kSums || R == 1, "the columns of a thread are one row's");
    __shared__ float slots[2][16];
    RowSum<TR> row_sum{slots};
    const int t = threadIdx.x % TR, H = a.H;
    const float mean = 1.0f / float(H);
    float acc[kSums ? 3 : 1][N][8];
    if constexpr (kSums) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][n][e] = 0.0f;
    }
    for (int64_t row = int64_t(blockIdx.x) * R + threadIdx.x / TR; row < a.T; row += int64_t(gridDim.x) * R) {
        const int64_t base = row * H;
        u32x4 dw[N], rw[N], ow[N], gw[N], hw[N];
        u32x2 cw[N];
        float cs[N];
        float g[N][8], b[N][8];
#pragma unroll
        for (int n = 0; n < N; ++n) dw[n] = load_octet<kRagged>(a.dn[0] + base, 8 * (n * TR + t), H);
        if (a.codes) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at = 8 * (n * TR + t);
                cw[n] = at < H ? *reinterpret_cast<const u32x2*>(a.codes + base + at) : u32x2{0, 0};
                cs[n] = at < H ? a.n_scale[(base + at) >> 6] : 0.0f;
            }
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) hw[n] = load_octet<kRagged>(a.h + base, 8 * (n * TR + t), H);
        }
        if (a.dres) {
#pragma unroll
            for (int n = 0; n < N; ++n) rw[n] = load_octet<kRagged>(a.dres + base, 8 * (n * TR + t), H);
        }
        if (a.o) {
#pragma unroll
            for (int n = 0; n < N; ++n) ow[n] = load_octet<kRagged>(a.o + base, 8 * (n * TR + t), H);
        }
        if (a.gate_kind != NF4_GATE_NONE) {
            const uint16_t* gate = a.gate + (a.gate_kind == NF4_GATE_TOKEN ? base : 0);
#pragma unroll
            for (int n = 0; n < N; ++n) gw[n] = load_octet<kRagged>(gate, 8 * (n * TR + t), H);
        }
        const float r = a.rstd[row], r_o = a.post ? a.rstd_o[row] : 1.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) unpack_octet(dw[n], g[n]);
        for (int i = 1; i < a.n_dn; ++i) {
            const uint16_t* more = (i == 1 ? a.dn[1] : a.dn[2]) + base;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float d[8];
                unpack_octet(load_octet<kRagged>(more, 8 * (n * TR + t), H), d);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[n][e] += d[e];
            }
        }
        if (a.codes) {
#pragma unroll
            for (int n = 0; n < N; ++n) act8_values8(cw[n], cs[n], b[n]);
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                unpack_octet(hw[n], b[n]);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[n][e] *= r;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float f[8];
            gain_octet<kRagged>(a.gain, a.offset, 8 * (n * TR + t), H, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (kSums) acc[0][n][e] = __builtin_fmaf(g[n][e], b[n][e], acc[0][n][e]);
                g[n][e] *= f[e];
                dot = __builtin_fmaf(g[n][e], b[n][e], dot);
            }
        }
        const float c = row_sum(dot) * mean;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float d[8];
            if (a.dres) {
                unpack_octet(rw[n], d);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) g[n][e] = __builtin_fmaf(r, __builtin_fmaf(-b[n][e], c, g[n][e]), d[e]);  // ds
            store_octet<kRagged>(a.dh + base, 8 * (n * TR + t), H, pack_octet(g[n]));
        }
        if (!a.d_o && !a.dgate_rows && !(kSums && (a.sums & 6))) continue;  // uniform
        // from here on g is dv, and b is u
        dot = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = 8 * (n * TR + t);
            float f[8], gate[8];
            if (a.o) {
                unpack_octet(ow[n], b[n]);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[n][e] *= r_o;
            }
            if (a.post) gain_octet<kRagged>(a.post_gain, a.offset, at, H, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[n][e] *= a.scale;
            if (a.gate_kind != NF4_GATE_NONE) {
                unpack_octet(gw[n], gate);
                if (a.dgate_rows || (kSums && (a.sums & 4))) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = g[n][e] * (a.post ? b[n][e] * f[e] : b[n][e]);
                    if (a.dgate_rows) store_octet<kRagged>(a.dgate_rows + base, at, H, pack_octet(x));
                    if constexpr (kSums) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[2][n][e] += x[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[n][e] *= gate[e];
            }
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (kSums) acc[1][n][e] = __builtin_fmaf(g[n][e], b[n][e], acc[1][n][e]);
                    g[n][e] *= f[e];
                    dot = __builtin_fmaf(g[n][e], b[n][e], dot);
                }
            }
        }
        if (!a.d_o) continue;
        if (a.post) {
            const float c_o = row_sum(dot) * mean;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[n][e] = r_o * __builtin_fmaf(-b[n][e], c_o, g[n][e]);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) store_octet<kRagged>(a.d_o + base, 8 * (n * TR + t), H, pack_octet(g[n]));
    }
    if constexpr (kSums) {
        // the partial rows are whole and aligned (pitch: octets)
        const int64_t pitch = int64_t((H + 7) / 8) * 8;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (!(a.sums >> i & 1)) continue;
            float* p = a.part + (int64_t(blockIdx.x) * 3 + i) * pitch;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at = 8 * (n * TR + t);
                if (at >= H) continue;
                *reinterpret_cast<f32x4*>(p + at) = f32x4{acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]};
                *reinterpret_cast<f32x4*>(p + at + 4) = f32x4{acc[i][n][4], acc[i][n][5], acc[i][n][6], acc[i][n][7]};
            }
        }
    }
}

struct SumArgs {
    const float* part;
    float* out[3];
    int groups, H;
};

// out[i][column] = the workgroups' sums: 64 columns a workgroup, its four waves a quarter of the
// workgroups each, in order.
__global__ __launch_bounds__(256) void k_residual_norm_sums(SumArgs a) {
    __shared__ float share[4][64];
    float* out = blockIdx.y == 0 ? a.out[0] : blockIdx.y == 1 ? a.out[1] : a.out[2];
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = int(blockIdx.x) * 64 + lane;
    const int64_t pitch = int64_t((a.H + 7) / 8) * 8;
    const int g0 = int(int64_t(a.groups) * wave / 4), g1 = int(int64_t(a.groups) * (wave + 1) / 4);
    float s = 0.0f;
    if (col < a.H) {
        const float* p = a.part + int64_t(blockIdx.y) * pitch + col;
#pragma unroll 8
        for (int g = g0; g < g1; ++g) s += p[int64_t(g) * 3 * pitch];
    }
    share[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < a.H) out[col] = ((share[0][lane] + share[1][lane]) + share[2][lane]) + share[3][lane];
}

// Threads a row and octets a thread.
struct Split {
    int threads, octets;
};

Split split_of(int64_t H) {
    if (H <= 512) return {64, 1};
    if (H <= 2048) return {256, 1};
    if (H <= 4096) return {256, 2};
    if (H <= 8192) return {256, 4};
    return {1024, 2};
}

// With sums over rows a thread holds three more values a column.
Split split_of_sums(int64_t H) {
    if (H <= 2048) return {256, 1};
    if (H <= 4096) return {512, 1};
    if (H <= 8192) return {1024, 1};
    return {1024, 2};
}

int64_t sum_groups(int64_t T, int64_t H) {
    const int64_t most = 262144 / split_of_sums(H).threads;  // half of what the card holds at once
    return std::min(T, most);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(const char* fn, int64_t T, int64_t H, int post_norm, const uint16_t* post_gain, int gate_kind,
                const uint16_t* gate, bool has_o, float scale, float gain_offset) {
    if (T < 0 || T > (int64_t(1) << 23) || H < 1 || H > kMaxWidth)
        return fail(NF4_E_SHAPE, "%s: need 0 <= T <= 2^23, 1 <= H <= 16384 (got T=%lld H=%lld)", fn, (long long)T, (long long)H);
    if (post_norm != 0 && post_norm != 1) return fail(NF4_E_ARG, "%s: post_norm must be 0 or 1 (got %d)", fn, post_norm);
    if (gate_kind < NF4_GATE_NONE || gate_kind > NF4_GATE_TOKEN)
        return fail(NF4_E_ARG, "%s: unknown gate_kind %d", fn, gate_kind);
    if (!std::isfinite(scale) || !std::isfinite(gain_offset))
        return fail(NF4_E_ARG, "%s: scale and gain_offset must be finite", fn);
    if (post_gain && !post_norm) return fail(NF4_E_ARG, "%s: post_gain without post_norm", fn);
    if ((gate != nullptr) != (gate_kind != NF4_GATE_NONE)) return fail(NF4_E_ARG, "%s: gate and gate_kind do not go together", fn);
    if (!has_o && (post_norm || gate)) return fail(NF4_E_ARG, "%s: post_norm and gate need a block's output", fn);
    return NF4_OK;
}

// Inputs and outputs with what they are called; outputs may meet nothing but, exactly, an input
// that `over` names (rows are read before they are written).
struct Buffers {
    const char* fn;
    ByteRange in[16], out[8];
    int n_in = 0, n_out = 0, status = NF4_OK;
    void take(ByteRange* to, int& n, const char* name, const void* p, size_t bytes, size_t align, bool need) {
        if (status != NF4_OK) return;
        if (!p && !need) return;
        if (!p || !aligned(p, align))
            status = fail(NF4_E_ARG, "%s: %s must be non-NULL and %zu-byte aligned", fn, name, align);
        to[n++] = {p, bytes};
    }
    void read(const char* name, const void* p, size_t bytes, size_t align, bool need) { take(in, n_in, name, p, bytes, align, need); }
    void write(const char* name, void* p, size_t bytes, size_t align, bool need) {
        take(out, n_out, name, p, bytes, align, need);
        if (status != NF4_OK || !p) return;
        const ByteRange& w = out[n_out - 1];
        for (int i = 0; i < n_out - 1; ++i)
            if (w.meets(out[i])) status = fail(NF4_E_ARG, "%s: %s overlaps another output", fn, name);
        for (int i = 0; i < n_in; ++i)
            if (w.meets(in[i])) status = fail(NF4_E_ARG, "%s: %s overlaps an input", fn, name);
    }
    // an output that may be one of the inputs a, b, c, d itself
    void write_over(const char* name, void* p, size_t bytes, bool need, const void* a, const void* b, const void* c, const void* d) {
        take(out, n_out, name, p, bytes, 2, need);
        if (status != NF4_OK || !p) return;
        const ByteRange& w = out[n_out - 1];
        for (int i = 0; i < n_out - 1; ++i)
            if (w.meets(out[i])) status = fail(NF4_E_ARG, "%s: %s overlaps another output", fn, name);
        for (int i = 0; i < n_in; ++i)
            if (w.meets(in[i]) && !(w.p == in[i].p && w.bytes == in[i].bytes && (p == a || p == b || p == c || p == d)))
                status = fail(NF4_E_ARG, "%s: %s overlaps an input", fn, name);
    }
};

template <int TR, int N>
void launch_fwd(const FwdArgs& a, bool ragged, hipStream_t s) {
    const dim3 grid(unsigned(std::min(cdiv(a.T, kRowsOf<TR>), kMaxGrid)));
    if (ragged)
        hipLaunchKernelGGL((k_residual_norm_fwd<TR, N, true>), grid, dim3(kBlock<TR>), 0, s, a);
    else
        hipLaunchKernelGGL((k_residual_norm_fwd<TR, N, false>), grid, dim3(kBlock<TR>), 0, s, a);
}

template <int TR, int N, bool kSums>
void launch_bwd(const BwdArgs& a, int64_t groups, bool ragged, hipStream_t s) {
    const dim3 grid(unsigned(kSums ? groups : std::min(cdiv(a.T, kRowsOf<TR>), kMaxGrid)));
    if (ragged)
        hipLaunchKernelGGL((k_residual_norm_bwd<TR, N, true, kSums>), grid, dim3(kBlock<TR>), 0, s, a);
    else
        hipLaunchKernelGGL((k_residual_norm_bwd<TR, N, false, kSums>), grid, dim3(kBlock<TR>), 0, s, a);
}

}  // namespace

}  // namespace nf4

using namespace nf4;

extern "C" int nf4_residual_norm_fwd(const uint16_t* h, const uint16_t* o, int64_t T, int64_t H, int post_norm,
                                     const uint16_t* post_gain, int gate_kind, const uint16_t* gate, float scale,
                                     const uint16_t* gain, float gain_offset, float eps, uint16_t* h_out, uint16_t* n,
                                     uint8_t* n_codes, float* n_scale, float* rstd_o, float* rstd, nf4_stream stream) {
    const char* fn = "nf4_residual_norm_fwd";
    const int st = check_sizes(fn, T, H, post_norm, post_gain, gate_kind, gate, o != nullptr || T == 0, scale, gain_offset);
    if (st != NF4_OK) return st;
    if (!std::isfinite(eps) || eps < 0.0f) return fail(NF4_E_ARG, "%s: eps must be finite and >= 0", fn);
    if ((n_codes != nullptr) != (n_scale != nullptr)) return fail(NF4_E_ARG, "%s: n_codes and n_scale go together", fn);
    if (n_codes && H % NF4_BLOCK != 0)
        return fail(NF4_E_SHAPE, "%s: a checkpoint needs H a multiple of %d (got %lld)", fn, NF4_BLOCK, (long long)H);
    if (T == 0) return NF4_OK;
    const size_t rows = size_t(T) * 4, one = size_t(H) * 2, all = size_t(T) * one;
    Buffers b{fn};
    b.read("h", h, all, 2, true);
    b.read("o", o, all, 2, false);
    b.read("post_gain", post_gain, one, 2, false);
    b.read("gain", gain, one, 2, false);
    b.read("gate", gate, gate_kind == NF4_GATE_TOKEN ? all : one, 2, false);
    if (h_out && !o) return fail(NF4_E_ARG, "%s: h_out without a block's output (h itself is the stream)", fn);
    b.write_over("h_out", h_out, all, o != nullptr, h, o, nullptr, nullptr);
    b.write_over("n", n, all, true, h, o, nullptr, nullptr);
    b.write("n_codes", n_codes, all / 2, 16, false);
    b.write("n_scale", n_scale, all / 32, 4, false);
    b.write("rstd_o", post_norm ? rstd_o : nullptr, rows, 4, post_norm);
    b.write("rstd", rstd, rows, 4, true);
    if (b.status != NF4_OK) return b.status;
    bool ragged = H % 8 != 0;
    for (const void* p : {(const void*)h, (const void*)o, (const void*)post_gain, (const void*)gate, (const void*)gain,
                          (const void*)h_out, (const void*)n})
        ragged = ragged || !aligned(p, 16);
    const FwdArgs a{h, o, post_gain, gate, gain, h_out, n, n_codes, n_scale, rstd_o, rstd, T, int(H), post_norm, gate_kind,
                    scale, gain_offset, eps};
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (const Split p = split_of(H); p.threads * 8 + p.octets) {
        case 64 * 8 + 1: launch_fwd<64, 1>(a, ragged, s); break;
        case 256 * 8 + 1: launch_fwd<256, 1>(a, ragged, s); break;
        case 256 * 8 + 2: launch_fwd<256, 2>(a, ragged, s); break;
        case 256 * 8 + 4: launch_fwd<256, 4>(a, ragged, s); break;
        default: launch_fwd<1024, 2>(a, ragged, s); break;
    }
    return check_launch(fn);
}

extern "C" size_t nf4_residual_norm_bwd_workspace(int64_t T, int64_t H, int sums) {
    if (T <= 0 || T > (int64_t(1) << 23) || H < 1 || H > kMaxWidth || !sums) return 0;
    return align256(size_t(sum_groups(T, H)) * 3 * size_t((H + 7) / 8 * 8) * 4);
}

extern "C" int nf4_residual_norm_bwd(const uint16_t* const* dn, int n_dn, const uint16_t* dres, const uint16_t* h,
                                     const uint8_t* n_codes, const float* n_scale, const float* rstd, const uint16_t* o,
                                     const float* rstd_o, int64_t T, int64_t H, int post_norm, const uint16_t* post_gain,
                                     int gate_kind, const uint16_t* gate, float scale, const uint16_t* gain,
                                     float gain_offset, uint16_t* dh, uint16_t* d_o, void* dgate, float* dpost_gain,
                                     float* dgain, void* ws, size_t ws_bytes, nf4_stream stream) {
    const char* fn = "nf4_residual_norm_bwd";
    const int st = check_sizes(fn, T, H, post_norm, post_gain, gate_kind, gate, true, scale, gain_offset);
    if (st != NF4_OK) return st;
    if (n_dn < 1 || n_dn > 3 || !dn) return fail(NF4_E_ARG, "%s: need 1 to 3 gradients dn (got %d)", fn, n_dn);
    if ((n_codes != nullptr) != (n_scale != nullptr)) return fail(NF4_E_ARG, "%s: n_codes and n_scale go together", fn);
    if (T > 0 && (h != nullptr) == (n_codes != nullptr))
        return fail(NF4_E_ARG, "%s: exactly one of h and the checkpoint of n is needed", fn);
    if (n_codes && gain)
        return fail(NF4_E_ARG, "%s: a checkpoint of n stands in for the normalised stream only without a gain", fn);
    if (n_codes && H % NF4_BLOCK != 0)
        return fail(NF4_E_SHAPE, "%s: a checkpoint needs H a multiple of %d (got %lld)", fn, NF4_BLOCK, (long long)H);
    if (dgate && gate_kind == NF4_GATE_NONE) return fail(NF4_E_ARG, "%s: dgate without a gate", fn);
    if (dpost_gain && !post_gain) return fail(NF4_E_ARG, "%s: dpost_gain without post_gain", fn);
    if (dgain && !gain) return fail(NF4_E_ARG, "%s: dgain without gain", fn);
    const bool channel = dgate && gate_kind == NF4_GATE_CHANNEL;
    const int sums = (dgain ? 1 : 0) | (dpost_gain ? 2 : 0) | (channel ? 4 : 0);
    const bool branch = d_o || dgate || dpost_gain, need_o = dgate || dpost_gain || (d_o && post_norm);
    const size_t rows = size_t(T) * 4, one = size_t(H) * 2, all = size_t(T) * one, need = nf4_residual_norm_bwd_workspace(T, H, sums);
    Buffers b{fn};
    if (T > 0) {
        for (int i = 0; i < n_dn; ++i) b.read("dn", dn[i], all, 2, true);
        b.read("dres", dres, all, 2, false);
        b.read("h", h, all, 2, false);
        b.read("n_codes", n_codes, all / 2, 16, false);
        b.read("n_scale", n_scale, all / 32, 4, false);
        b.read("rstd", rstd, rows, 4, true);
        b.read("o", o, all, 2, need_o);
        b.read("rstd_o", rstd_o, rows, 4, branch && post_norm);
    }
    b.read("post_gain", post_gain, one, 2, false);
    b.read("gate", gate, gate_kind == NF4_GATE_TOKEN ? all : one, 2, false);
    b.read("gain", gain, one, 2, false);
    b.write_over("dh", dh, all, T > 0, dres, dn[0], n_dn > 1 ? dn[1] : nullptr, n_dn > 2 ? dn[2] : nullptr);
    b.write_over("d_o", d_o, all, false, o, dn[0], n_dn > 1 ? dn[1] : nullptr, n_dn > 2 ? dn[2] : nullptr);
    b.write("dgate", dgate, channel ? size_t(H) * 4 : all, channel ? 4 : 2, false);
    b.write("dpost_gain", dpost_gain, size_t(H) * 4, 4, false);
    b.write("dgain", dgain, size_t(H) * 4, 4, false);
    if (need) {
        if (b.status == NF4_OK && (!ws || ws_bytes < need || !aligned(ws, 256)))
            return fail(NF4_E_ARG, "%s: workspace of %zu bytes (256-byte aligned) needed for T=%lld H=%lld, got %zu", fn, need,
                        (long long)T, (long long)H, ws_bytes);
        b.write("ws", ws, need, 256, true);
    }
    if (b.status != NF4_OK) return b.status;
    bool ragged = H % 8 != 0;
    for (const void* p : {(const void*)dn[0], n_dn > 1 ? (const void*)dn[1] : nullptr, n_dn > 2 ? (const void*)dn[2] : nullptr,
                          (const void*)dres, (const void*)h, (const void*)o, (const void*)post_gain, (const void*)gate,
                          (const void*)gain, (const void*)dh, (const void*)d_o, channel ? nullptr : (const void*)dgate})
        ragged = ragged || !aligned(p, 16);
    BwdArgs a{};
    for (int i = 0; i < n_dn; ++i) a.dn[i] = dn[i];
    a.dres = dres, a.h = h, a.post_gain = post_gain, a.gain = gain, a.codes = n_codes, a.n_scale = n_scale, a.rstd = rstd;
    a.o = need_o ? o : nullptr, a.rstd_o = rstd_o, a.dh = dh, a.d_o = d_o, a.part = static_cast<float*>(ws), a.sums = sums;
    a.dgate_rows = channel ? nullptr : static_cast<uint16_t*>(dgate);
    // the branch's gate is not read where nothing of the branch is wanted
    a.gate_kind = branch ? gate_kind : NF4_GATE_NONE, a.gate = gate, a.post = branch && post_norm, a.T = T, a.H = int(H);
    a.n_dn = n_dn, a.scale = scale, a.offset = gain_offset;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t groups = T > 0 ? sum_groups(T, H) : 0;
    if (T > 0 && sums) {
        switch (const Split p = split_of_sums(H); p.threads * 8 + p.octets) {
            case 256 * 8 + 1: launch_bwd<256, 1, true>(a, groups, ragged, s); break;
            case 512 * 8 + 1: launch_bwd<512, 1, true>(a, groups, ragged, s); break;
            case 1024 * 8 + 1: launch_bwd<1024, 1, true>(a, groups, ragged, s); break;
            default: launch_bwd<1024, 2, true>(a, groups, ragged, s); break;
        }
    } else if (T > 0) {
        switch (const Split p = split_of(H); p.threads * 8 + p.octets) {
            case 64 * 8 + 1: launch_bwd<64, 1, false>(a, 0, ragged, s); break;
            case 256 * 8 + 1: launch_bwd<256, 1, false>(a, 0, ragged, s); break;
            case 256 * 8 + 2: launch_bwd<256, 2, false>(a, 0, ragged, s); break;
            case 256 * 8 + 4: launch_bwd<256, 4, false>(a, 0, ragged, s); break;
            default: launch_bwd<1024, 2, false>(a, 0, ragged, s); break;
        }
    }
    if (sums) {
        const SumArgs q{a.part, {dgain, dpost_gain, channel ? static_cast<float*>(dgate) : nullptr}, int(groups), int(H)};
        hipLaunchKernelGGL(k_residual_norm_sums, dim3(unsigned(cdiv(H, 64)), 3), dim3(256), 0, s, q);
    }
    return check_launch(fn);
}
