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
// Measured, calls in a row, 8192 x 8192 (what it has to move): norm alone 46 us (5.8 TB/s), add 88 (6.1), both norms, a gate
// a channel and the checkpoint 97-103 (6.3-5.9; 101-106 in a kernel trace); backward of one reader 87 (6.2), both norms, a gate a token, three readers
// and the gains' sums 233 (5.8). 4096 x 16384 the same 269 (5.0), 4096 x 3583 80 (3.7), 2731 x 5120 60 (4.6).
#include <cmath>

#include "../../include/nf4lora.h"
#include "act8.h"
#include "common.h"

namespace nf4 {

namespace {

constexpr size_t kLastLevelCache = size_t(256) << 20;
constexpr int64_t kMaxWidth = 16384;
constexpr int64_t kMaxGrid = int64_t(1) << 21;  // workgroups; rows past it are looped over

// A row belongs to a wave (kWave: widths up to 512, four rows a workgroup) or to a workgroup of as
// many waves as its octets need at N octets a thread: octet n of thread t is at column 8 (n TR + t).
template <bool kWave>
struct Place {
    int t, TR, first, step;  // the thread within its row's TR; the first row and the step to the next
    __device__ __forceinline__ Place()
        : t(kWave ? threadIdx.x & 63 : threadIdx.x), TR(kWave ? 64 : blockDim.x),
          first(kWave ? __builtin_amdgcn_readfirstlane(int(blockIdx.x) * 4 + (threadIdx.x >> 6)) : blockIdx.x),
          step(gridDim.x * (kWave ? 4 : 1)) {}
    __device__ __forceinline__ int at(int n) const { return 8 * (n * TR + t); }
};

// A thread's octets of one row, zeros past its end. Rows of whole, aligned 16-byte pieces go through
// a descriptor over the row, which also stands for an absent tensor (p NULL: zeros, nothing stored)
// without a branch, so that the loads of a row are issued back to back. kRagged: any others, by loads at
// 2-byte alignment that stay within the row: octets that pass its end are loaded from its last whole one, and
// `settle` moves them into place, later, where they are used (with a branch at each octet that is not whole, and
// elements loaded one by one, 4096 x 3583 backward with everything takes 185 us instead of 80).
struct __attribute__((packed, aligned(2))) LooseOctet {
    u32x4 w;
};

template <bool kRagged, bool kStream = false, int N, bool kWave>
__device__ __forceinline__ void load_line(const uint16_t* p, int64_t base, int H, const Place<kWave>& pl, u32x4 (&x)[N]) {
    if constexpr (!kRagged) {
        const auto r = make_rsrc(p ? p + base : nullptr, p ? uint32_t(H) * 2u : 0u);
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = kStream ? buf_load16_nt(r, uint32_t(pl.at(n)) * 2u) : buf_load16(r, uint32_t(pl.at(n)) * 2u);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = u32x4{0, 0, 0, 0};
        if (!p) return;
        if (H >= 8) {
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] = reinterpret_cast<const LooseOctet*>(p + base + min(pl.at(n), H - 8))->w;
        } else if (pl.t == 0) {  // a row's elements where an octet that ends with it has them
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (e >= 8 - H) x[0][e / 2] |= uint32_t(p[base + e - (8 - H)]) << (16 * (e % 2));
        }
    }
}

template <bool kRagged, int N, bool kWave>
__device__ __forceinline__ void settle(int H, const Place<kWave>& pl, u32x4 (&x)[N]) {
    if constexpr (!kRagged) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int by = max(0, pl.at(n) - (H - 8));  // elements that lie before the octet
        if (!__ballot(by > 0)) continue;
        u32x4 y = x[n];
        if (by & 2) y = u32x4{y[1], y[2], y[3], 0};
        if (by & 4) y = u32x4{y[2], y[3], 0, 0};
        if (by & 1)
            y = u32x4{__builtin_amdgcn_alignbit(y[1], y[0], 16), __builtin_amdgcn_alignbit(y[2], y[1], 16),
                      __builtin_amdgcn_alignbit(y[3], y[2], 16), y[3] >> 16};
        x[n] = by >= 8 ? u32x4{0, 0, 0, 0} : y;
    }
}

template <bool kRagged, int N, bool kWave>
__device__ __forceinline__ void store_line(uint16_t* p, int64_t base, int H, const Place<kWave>& pl, const u32x4 (&x)[N]) {
    if constexpr (!kRagged) {
        const auto r = make_rsrc(p ? p + base : nullptr, p ? uint32_t(H) * 2u : 0u);
#pragma unroll
        for (int n = 0; n < N; ++n) __builtin_amdgcn_raw_buffer_store_b128(x[n], r, pl.at(n) * 2, 0, 2);
    } else {
        if (!p) return;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = pl.at(n);
            if (at + 8 <= H) {
                reinterpret_cast<LooseOctet*>(p + base + at)->w = x[n];
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e < H) p[base + at + e] = uint16_t(x[n][e / 2] >> (16 * (e % 2)));
        }
    }
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

// Threads of a workgroup by the widths it takes: 256, a wave a row, up to 512 elements; up to 512, a row
// of at most 8192; up to 1024 for wider ones.
constexpr int kWaveRows = 256, kRows = 512, kWideRows = 1024;
// With a branch's sums over rows, wide rows take four octets a thread of half as many threads: what a thread holds
// besides its octets it holds once (1024 x 12288, gains and a gate a channel, 57 us against 62 at two, a gate a token
// and three readers 69 against 79; 4096 x 16384 193 against 201, 269 against 275).
constexpr int kManyOctets = 4;
__host__ __device__ constexpr int threads_of(int kind, int octets) { return octets == kManyOctets ? kind / 2 : kind; }
constexpr int kMaxWaves = 16;  // of a workgroup

// Sum over a row's threads - a wave's lanes, or the whole workgroup - in a fixed order. Two slots
// taken in turn need one barrier a sum: whoever writes a slot again has met the barrier that
// followed its last reads.
template <bool kWave>
struct RowSum {
    float (&slots)[2][kMaxWaves];
    int turn = 0;
    __device__ __forceinline__ explicit RowSum(float (&s)[2][kMaxWaves]) : slots(s) {
        // places without a wave add zeros; the first sum's barrier comes before its reads
        const int i = threadIdx.x, waves = blockDim.x >> 6;
        if (!kWave && i < kMaxWaves && i >= waves) slots[0][i] = slots[1][i] = 0.0f;
    }
    __device__ __forceinline__ float operator()(float v) {
        v = lane_sum(v);
        if constexpr (kWave) return v;
        float(&slot)[kMaxWaves] = slots[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxWaves; i += 4) s += (slot[i] + slot[i + 1]) + (slot[i + 2] + slot[i + 3]);
        return s;
    }
};

struct FwdArgs {
    const uint16_t *h, *o, *post_gain, *gate, *gain;
    uint16_t *h_out, *n;
    uint8_t* codes;
    float *n_scale, *rstd_o, *rstd;
    int T, H, gate_kind, stream;
    float scale, offset, eps;
};

// A gain's factors, 1 without one.
__device__ __forceinline__ void gain_octet(bool has, u32x4 w, float offset, float (&f)[8]) {
    unpack_octet(w, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = has ? f[e] + offset : 1.0f;
}

// kBlock: 0 the norm alone, 1 a block's output joins, 2 it is normalised first. With many rows a
// workgroup takes several, the next one's loads under way while a row is reduced.
template <int N, bool kRagged, int kThreads, int kBlock>
__global__ __launch_bounds__(kThreads) void k_residual_norm_fwd(FwdArgs a) {
    constexpr bool kWave = kThreads == kWaveRows;
    constexpr bool kAhead = kBlock > 1;
    __shared__ float slots[2][kMaxWaves];
    RowSum<kWave> row_sum(slots);
    const Place<kWave> p;
    const int H = a.H;
    const float mean = 1.0f / float(H);
    struct {
        u32x4 o[kBlock ? N : 1], h[N], gate[kBlock ? N : 1];
    } next;
    auto load_as = [&](int row, auto stream) {  // in the order of their use
        constexpr bool kStream = decltype(stream)::value;
        const int64_t base = int64_t(row) * H;
        if constexpr (kBlock > 0) load_line<kRagged, kStream>(a.o, base, H, p, next.o);
        load_line<kRagged, kStream>(a.h, base, H, p, next.h);
        if constexpr (kBlock > 0) load_line<kRagged>(a.gate, a.gate_kind == NF4_GATE_TOKEN ? base : 0, H, p, next.gate);
    };
    auto load = [&](int row) { a.stream ? load_as(row, std::true_type{}) : load_as(row, std::false_type{}); };
    u32x4 fw[N], pw[kBlock > 1 ? N : 1];  // the same for all rows
    if (p.first < a.T) load(p.first);
    if constexpr (kBlock > 1) load_line<kRagged>(a.post_gain, 0, H, p, pw), settle<kRagged>(H, p, pw);
    load_line<kRagged>(a.gain, 0, H, p, fw);
    settle<kRagged>(H, p, fw);
    for (int row = p.first; row < a.T; row += p.step) {
        const int64_t base = int64_t(row) * H;
        if (!kAhead && row != p.first) load(row);
        auto in = next;
        if constexpr (kBlock > 0) settle<kRagged>(H, p, in.o), settle<kRagged>(H, p, in.gate);
        settle<kRagged>(H, p, in.h);
        u32x4 out[N];
        if (kAhead && row + p.step < a.T) load(row + p.step);
        float s[N][8];
        if constexpr (kBlock > 0) {
            float r = 1.0f;
            if constexpr (kBlock > 1) {
                float ss = 0.0f;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float v[8];
                    unpack_octet(in.o[n], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
                }
                r = 1.0f / sqrtf(row_sum(ss) * mean + a.eps);
                if (p.t == 0) a.rstd_o[row] = r;
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float v[8], f[8];
                unpack_octet(in.h[n], s[n]);
                unpack_octet(in.o[n], v);
                if constexpr (kBlock > 1) {
                    gain_octet(a.post_gain != nullptr, pw[n], a.offset, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = v[e] * r * f[e];
                }
                if (a.gate_kind != NF4_GATE_NONE) {
                    unpack_octet(in.gate[n], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= f[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s[n][e] = __builtin_fmaf(a.scale, v[e], s[n][e]);
                out[n] = pack_octet(s[n]);
            }
            store_line<kRagged>(a.h_out, base, H, p, out);
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) unpack_octet(in.h[n], s[n]);
        }
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(s[n][e], s[n][e], ss);
        const float r = 1.0f / sqrtf(row_sum(ss) * mean + a.eps);
        if (p.t == 0) a.rstd[row] = r;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float f[8];
            gain_octet(a.gain != nullptr, fw[n], a.offset, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s[n][e] * r;
            out[n] = pack_octet(f);
        }
        store_line<kRagged>(a.n, base, H, p, out);
        if (a.codes) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at = p.at(n);
                if (at >= H) continue;  // H % 64 == 0: the 8 lanes of a block are all in or all out
                float step;
                *reinterpret_cast<u32x2*>(a.codes + base + at) = act8_quantize8(out[n], step);
                if ((p.t & 7) == 0) a.n_scale[(base + at) >> 6] = step;
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
    int T, H, n_dn, gate_kind, stream;
    float scale, offset;
};

// A row's inputs as loaded.
template <int N, int kBranch>
struct RowIn {
    u32x4 d[3][N], h[N], res[N];  // h: bf16, or two dwords of codes and their scale
    u32x4 o[kBranch ? N : 1], gate[kBranch ? N : 1];
    float r, r_o;
};

template <int N, bool kRagged, bool kStream, int kBranch, bool kWave>
__device__ __forceinline__ void load_row_as(const BwdArgs& a, const Place<kWave>& p, int row, RowIn<N, kBranch>& in) {
    const int64_t base = int64_t(row) * a.H;
    const int H = a.H;
#pragma unroll
    for (int i = 0; i < 3; ++i) load_line<kRagged, kStream>(a.dn[i], base, H, p, in.d[i]);
    if (a.codes) {
        const auto rc = make_rsrc(a.codes + base, uint32_t(H));
        const auto rs = make_rsrc(a.n_scale + int64_t(row) * (H / 64), uint32_t(H / 64) * 4u);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const u32x2 c = kStream ? buf_load8_nt(rc, uint32_t(p.at(n))) : buf_load8(rc, uint32_t(p.at(n)));
            in.h[n] = u32x4{c.x, c.y, buf_load_u32(rs, uint32_t(p.at(n)) / 64 * 4u), 0};
        }
    } else {
        load_line<kRagged, kStream>(a.h, base, H, p, in.h);
    }
    in.r = a.rstd[row];
    load_line<kRagged, kStream>(a.dres, base, H, p, in.res);
    if constexpr (kBranch > 0) {
        load_line<kRagged, kStream>(a.o, base, H, p, in.o);
        load_line<kRagged>(a.gate, a.gate_kind == NF4_GATE_TOKEN ? base : 0, H, p, in.gate);
        in.r_o = kBranch > 1 ? a.rstd_o[row] : 1.0f;
    }
}

template <int N, bool kRagged, int kBranch, bool kWave>
__device__ __forceinline__ void load_row(const BwdArgs& a, const Place<kWave>& p, int row, RowIn<N, kBranch>& in) {
    if (a.stream)
        load_row_as<N, kRagged, true>(a, p, row, in);
    else
        load_row_as<N, kRagged, false>(a, p, row, in);
}

// kBranch: gradients of the block's side are wanted, 2 with its norm. kSums: sums over rows are; a
// workgroup then takes many rows, and (but for wide ones, which fill the registers) the next row's loads are
// under way while a row is reduced. kRowKind: kWaveRows, kRows or kWideRows.
template <int N, bool kRagged, int kRowKind, int kBranch, bool kSums>
__global__ __launch_bounds__(threads_of(kRowKind, N)) void k_residual_norm_bwd(BwdArgs a) {
    constexpr bool kWave = kRowKind == kWaveRows, kWide = kRowKind == kWideRows;
    constexpr int kThreads = threads_of(kRowKind, N);
    constexpr bool kAhead = (kSums || kBranch > 1) && !kWide;
    constexpr int kKinds = !kSums ? 1 : kBranch ? 3 : 1;
    __shared__ float slots[2][kMaxWaves];
    RowSum<kWave> row_sum(slots);
    const Place<kWave> p;
    const int H = a.H;
    const float mean = 1.0f / float(H);
    // the sums over rows: dgain, and with a branch dpost_gain and dgate. Of wide rows the latter two are
    // kept in LDS
    constexpr bool kInLds = kKinds > 1 && kWide;
    constexpr int kHeld = kInLds ? 1 : kKinds;
    float acc[kHeld][N][8];
    __shared__ f32x4 wide[kInLds ? 2 * N * 2 * kThreads : 1];  // [kind][octet][half][thread]
    auto wide_at = [&](int kind, int n, int half) -> f32x4& {
        return wide[(((kind - 1) * N + n) * 2 + half) * kThreads + threadIdx.x];
    };
    auto add = [&](int kind, int n, const float (&x)[8]) {
        if constexpr (kInLds) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
                wide_at(kind, n, half) += f32x4{x[4 * half], x[4 * half + 1], x[4 * half + 2], x[4 * half + 3]};
        } else if constexpr (kSums) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[kind][n][e] += x[e];
        }
    };
    if constexpr (kSums) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][n][e] = 0.0f;
            if constexpr (kInLds) {
#pragma unroll
                for (int i = 0; i < 4; ++i) wide_at(1 + i / 2, n, i % 2) = f32x4{0, 0, 0, 0};
            }
        }
    }
    RowIn<N, kBranch> next;
    u32x4 fw[N], pw[kBranch > 1 ? N : 1];  // the same for all rows
    if (kAhead && p.first < a.T) load_row<N, kRagged>(a, p, p.first, next);
    auto load_gain = [&]() { load_line<kRagged>(a.gain, 0, H, p, fw), settle<kRagged>(H, p, fw); };
    auto load_post_gain = [&]() {
        if constexpr (kBranch > 1) load_line<kRagged>(a.post_gain, 0, H, p, pw), settle<kRagged>(H, p, pw);
    };
    if constexpr (!kInLds) load_gain(), load_post_gain();
    for (int row = p.first; row < a.T; row += p.step) {
        const int64_t base = int64_t(row) * H;
        if constexpr (!kAhead) load_row<N, kRagged>(a, p, row, next);
        // where registers are short the gains stay packed: made opaque here, their factors are not formed once, before
        // the rows (2000 x 7001, gains and a gate a channel, 83 us, spilling, for 63; 8192 x 8192, which does not
        // spill, 149 us for 156 without this)
        if constexpr (kRagged && kAhead && kSums && kBranch > 1 && N > 1) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(fw[n][i]), "+v"(pw[n][i]));
        }
        RowIn<N, kBranch> in = next;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < a.n_dn) settle<kRagged>(H, p, in.d[i]);
        if (!a.codes) settle<kRagged>(H, p, in.h);
        settle<kRagged>(H, p, in.res);
        if constexpr (kBranch > 0) settle<kRagged>(H, p, in.o), settle<kRagged>(H, p, in.gate);
        float g[N][8], b[N][8];
        u32x4 out[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float d[8];
            unpack_octet(in.d[0][n], g[n]);
#pragma unroll
            for (int i = 1; i < 3; ++i) {
                if (i >= a.n_dn) continue;
                unpack_octet(in.d[i][n], d);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[n][e] += d[e];
            }
            if (a.codes) {
                act8_values8(u32x2{in.h[n][0], in.h[n][1]}, __uint_as_float(in.h[n][2]), b[n]);
            } else {
                unpack_octet(in.h[n], b[n]);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[n][e] *= in.r;
            }
        }
        if (kAhead && row + p.step < a.T) load_row<N, kRagged>(a, p, row + p.step, next);
        // gains of wide rows where they are used: held over the rows, and unpacked there, they overflow the
        // registers (4096 x 16384, gains and a gate a channel, 464 us)
        if constexpr (kInLds) load_gain();
        float dot = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float f[8];
            gain_octet(a.gain != nullptr, fw[n], a.offset, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (kSums) acc[0][n][e] = __builtin_fmaf(g[n][e], b[n][e], acc[0][n][e]);
                g[n][e] *= f[e];
                dot = __builtin_fmaf(g[n][e], b[n][e], dot);
            }
        }
        if constexpr (kInLds) load_post_gain();
        const float c = row_sum(dot) * mean;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float d[8];
            unpack_octet(in.res[n], d);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[n][e] = __builtin_fmaf(in.r, __builtin_fmaf(-b[n][e], c, g[n][e]), d[e]);  // ds
            out[n] = pack_octet(g[n]);
        }
        store_line<kRagged>(a.dh, base, H, p, out);
        if constexpr (kBranch > 0) {
            // from here on g is dv, and b is u
            dot = 0.0f;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float f[8], x[8];
                unpack_octet(in.o[n], b[n]);
                if constexpr (kBranch > 1) {
                    gain_octet(a.post_gain != nullptr, pw[n], a.offset, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) b[n][e] *= in.r_o;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[n][e] *= a.scale;
                if (a.gate_kind != NF4_GATE_NONE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = g[n][e] * (kBranch > 1 ? b[n][e] * f[e] : b[n][e]);
                    if constexpr (kSums) add(2, n, x);
                    out[n] = pack_octet(x);
                    unpack_octet(in.gate[n], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[n][e] *= x[e];
                }
                if constexpr (kBranch > 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = g[n][e] * b[n][e];
                    if constexpr (kSums) add(1, n, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        g[n][e] *= f[e];
                        dot = __builtin_fmaf(g[n][e], b[n][e], dot);
                    }
                }
            }
            if (a.dgate_rows) store_line<kRagged>(a.dgate_rows, base, H, p, out);
            if constexpr (kBranch > 1) {
                const float c_o = row_sum(dot) * mean;
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[n][e] = in.r_o * __builtin_fmaf(-b[n][e], c_o, g[n][e]);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) out[n] = pack_octet(g[n]);
            store_line<kRagged>(a.d_o, base, H, p, out);
        }
    }
    if constexpr (kSums) {
        // the partial rows are whole and aligned (pitch: octets)
        const int64_t pitch = int64_t((H + 7) / 8) * 8;
        __shared__ float share[kWave ? 3 * 64 * 8 : 1];
#pragma unroll
        for (int i = 0; i < kKinds; ++i) {
            if (!(a.sums >> i & 1)) continue;
            const int k = kInLds ? 0 : i;
            if constexpr (kWave) {  // the workgroup's four waves, in order
                const int wave = threadIdx.x >> 6;
                __syncthreads();
                if (wave > 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) share[((wave - 1) * 8 + e) * 64 + p.t] = acc[k][0][e];
                }
                __syncthreads();
                if (wave > 0) continue;
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[k][0][e] += share[(w * 8 + e) * 64 + p.t];
            }
            float* q = a.part + (int64_t(blockIdx.x) * 3 + i) * pitch;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at = p.at(n);
                if (at >= H) continue;
                if constexpr (kInLds) {
                    if (i > 0) {
                        *reinterpret_cast<f32x4*>(q + at) = wide_at(i, n, 0);
                        *reinterpret_cast<f32x4*>(q + at + 4) = wide_at(i, n, 1);
                        continue;
                    }
                }
                *reinterpret_cast<f32x4*>(q + at) = f32x4{acc[k][n][0], acc[k][n][1], acc[k][n][2], acc[k][n][3]};
                *reinterpret_cast<f32x4*>(q + at + 4) = f32x4{acc[k][n][4], acc[k][n][5], acc[k][n][6], acc[k][n][7]};
            }
        }
    }
}

struct SumArgs {
    const float* part;
    float* out[3];
    int groups, H;
};

// out[i][column] = the workgroups' sums: 64 columns a workgroup, each of its waves a run of the
// workgroups, in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void k_residual_norm_sums(SumArgs a) {
    __shared__ float share[kSumWaves][64];
    float* out = blockIdx.y == 0 ? a.out[0] : blockIdx.y == 1 ? a.out[1] : a.out[2];
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = int(blockIdx.x) * 64 + lane;
    const int64_t pitch = int64_t((a.H + 7) / 8) * 8;
    const int g0 = a.groups * wave / kSumWaves, g1 = a.groups * (wave + 1) / kSumWaves;
    float s = 0.0f;
    if (col < a.H) {
        const float* p = a.part + int64_t(blockIdx.y) * pitch + col;
#pragma unroll 8
        for (int g = g0; g < g1; ++g) s += p[int64_t(g) * 3 * pitch];
    }
    share[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || col >= a.H) return;
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) s += share[w][lane];
    out[col] = s;
}

struct Split {
    int octets, kind, threads;  // octets a thread; kWaveRows, kRows or kWideRows; the workgroup's threads
};

Split split_of(int64_t H) {
    const int64_t all = cdiv(H, 8);
    if (all <= 64) return {1, kWaveRows, 256};
    const int n = all <= 512 ? 1 : 2;
    return {n, all <= 1024 ? kRows : kWideRows, int(cdiv(cdiv(all, n), 64) * 64)};
}

// Workgroups that sum over rows: eight waves a CU (at least one workgroup), which the next row's loads
// keep busy; more only add to the shares that the second kernel reads (8192 rows of 1024, gains and a
// gate a token: 4, 8, 16, 32 waves 45.7, 42.7, 49.9, 56.2 us). Two rows a workgroup at least once
// there are 128 of them.
int64_t sum_groups(int64_t T, int64_t H) {
    const Split p = split_of(H);
    const int64_t rows = p.kind == kWaveRows ? 4 : 1;
    const int64_t most = kChipCUs * std::max(1, 512 / p.threads);
    return std::min(std::max<int64_t>(cdiv(T, rows * 2), std::min<int64_t>(cdiv(T, rows), 128)), most);
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

// kernel<octets a thread, ragged, kind of rows>, picked by width and alignment.
template <int kWideOctets, template <int, bool, int> class Kernel, typename Args>
void launch(const Args& a, int64_t H, bool ragged, unsigned grid, hipStream_t s) {
    const Split p = split_of(H);
    const auto kernel =
        p.kind == kWaveRows   ? (ragged ? Kernel<1, true, kWaveRows>::get() : Kernel<1, false, kWaveRows>::get())
        : p.kind == kWideRows ? (ragged ? Kernel<kWideOctets, true, kWideRows>::get() : Kernel<kWideOctets, false, kWideRows>::get())
        : p.octets == 1       ? (ragged ? Kernel<1, true, kRows>::get() : Kernel<1, false, kRows>::get())
                              : (ragged ? Kernel<2, true, kRows>::get() : Kernel<2, false, kRows>::get());
    const int threads = p.kind == kWideRows ? int(cdiv(cdiv(H, 8 * kWideOctets), 64) * 64) : p.threads;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, s, a);
}

template <int kBlock>
struct Fwd {
    template <int N, bool kRagged, int kThreads>
    struct Kernel {
        static auto get() { return k_residual_norm_fwd<N, kRagged, kThreads, kBlock>; }
    };
};

template <int kBranch, bool kSums>
struct Bwd {
    template <int N, bool kRagged, int kThreads>
    struct Kernel {
        static auto get() { return k_residual_norm_bwd<N, kRagged, kThreads, kBranch, kSums>; }
    };
};

// Workgroups of a row, or of four rows of a wave each. loop: as many as the card holds.
unsigned rows_grid(int64_t T, int64_t H, bool loop, bool ragged) {
    const Split p = split_of(H);
    // (at two octets a thread of ragged rows the next row's loads cost registers: 2000 x 7001 47 -> 54 us; at one
    // they gain: 8192 x 1021, a gate a token, 21.4 -> 19.4)
    loop = loop && !(ragged && p.octets == 2);
    const int64_t most = loop ? (p.octets == 2 ? 131072 : 262144) / std::min(p.threads, kRows) : kMaxGrid;
    return unsigned(std::min(cdiv(T, p.kind == kWaveRows ? 4 : 1), most));
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
    const int large = all * (n_codes ? 5 : 4) / 2 * (o ? 2 : 1) > kLastLevelCache;
    const FwdArgs a{h, o, post_gain, gate, gain, h_out, n, n_codes, n_scale, rstd_o, rstd, int(T), int(H), gate_kind,
                    large, scale, gain_offset, eps};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const unsigned grid = rows_grid(T, H, post_norm, ragged);
    if (!o)
        launch<2, Fwd<0>::Kernel>(a, H, ragged, grid, s);
    else if (!post_norm)
        launch<2, Fwd<1>::Kernel>(a, H, ragged, grid, s);
    else
        launch<2, Fwd<2>::Kernel>(a, H, ragged, grid, s);
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
    a.gate_kind = branch ? gate_kind : NF4_GATE_NONE, a.gate = gate, a.T = int(T), a.H = int(H);
    a.n_dn = n_dn, a.stream = all * (n_dn + 3 + (branch ? 2 : 0)) > kLastLevelCache, a.scale = scale, a.offset = gain_offset;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t groups = T > 0 ? sum_groups(T, H) : 0;
    const unsigned grid = sums ? unsigned(groups) : rows_grid(T, H, branch && post_norm, ragged);
    const int kind = !branch ? 0 : post_norm ? 2 : 1;
    if (T > 0 && sums) {
        if (kind == 0)
            launch<2, Bwd<0, true>::Kernel>(a, H, ragged, grid, s);
        else if (kind == 1)
            launch<kManyOctets, Bwd<1, true>::Kernel>(a, H, ragged, grid, s);
        else
            launch<kManyOctets, Bwd<2, true>::Kernel>(a, H, ragged, grid, s);
    } else if (T > 0) {
        if (kind == 0)
            launch<2, Bwd<0, false>::Kernel>(a, H, ragged, grid, s);
        else if (kind == 1)
            launch<2, Bwd<1, false>::Kernel>(a, H, ragged, grid, s);
        else
            launch<2, Bwd<2, false>::Kernel>(a, H, ragged, grid, s);
    }
    if (sums) {
        const SumArgs q{a.part, {dgain, dpost_gain, channel ? static_cast<float*>(dgate) : nullptr}, int(groups), int(H)};
        hipLaunchKernelGGL(k_residual_norm_sums, dim3(unsigned(cdiv(H, 64)), 3), dim3(64 * kSumWaves), 0, s, q);
    }
    return check_launch(fn);
}
