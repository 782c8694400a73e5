// Grouped-query softmax attention over packed sequences, forward and backward, for the
// decoder stack's training step. With q [T][hq*D], k, v [T][hkv*D] in bf16, G = hq / hkv
// query heads per kv head, s = scale, and for row i of a sequence the keys j of the same
// sequence (j <= i when causal):
//   S_ij = s q_i . k_j      lse_i = log sum_j e^{S_ij}      o_i = sum_j e^{S_ij - lse_i} v_j
//   P = e^{S - lse}   delta_i = do_i . o_i   dS_ij = P_ij (do_i . v_j - delta_i)
//   dv_j = sum_i P_ij do_i   dq_i = s sum_j dS_ij k_j   dk_j = s sum_i dS_ij q_i
// (dk, dv also summed over the G query heads of a kv head). Scores are never stored: the
// backward recomputes P from lse. Everything is fp32 except the operands of the second
// products, which are P and dS rounded to bf16 for the bf16 MFMA: a relative error of at
// most 2^-8 per term, which leaves the results 1.40 to 1.45 times as far from exact (2-norm) as
// their own rounding does, at every length (evaluated in fp64 on the CPU, 2 to 512 rows of one
// head, q twice as long as k). In a short call, whose few errors do not average, a single result
// scatters far above that: 2 rows up to 3.6 times, 16 up to 2.1, 64 up to 1.65, 512 up to 1.5. dS
// is then the sum of two bf16 values, each multiplied (FINE below). What counts for that is a
// call's rows, not its sequences', so the same sequence rounds otherwise in a longer call.
//
// MFMA layout used throughout (32x32x16): an accumulator lane l holds column l % 32 and
// rows 8 (e / 4) + 4 (l / 32) + e % 4; an operand lane holds one row (or column) and 8
// contraction indices. Each first product is formed with the later contraction index as
// accumulator row, so that elements 8g .. 8g + 7 of the accumulator, rounded, are the
// lane's operand of the second product as they stand, with the contraction order
//   lane half h, slot j  <->  index 16 g + 8 (j / 4) + 4 h + j % 4,
// and the other operand is read from row-major LDS in that same order by two transposing
// reads (ds_read_b64_tr_b16). P and dS never cross lanes or go through LDS.
#include <cmath>

#include "../../include/nf4lora.h"
#include "common.h"
#include "device.h"

namespace nf4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKeyWaves = 4;  // blocks of 32 keys of a dk/dv workgroup
constexpr int64_t kMaxSeqs = int64_t(1) << 16;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) void* lds_ptr;

struct AttnArgs {
    const uint16_t *q, *k, *v, *o, *dO;
    const float* lse_in;
    uint16_t *out, *dq, *dk, *dv;
    float *lse, *stats, *part;  // stats [2][hq][T]: lse * log2 e, delta; part: fp32 shares of dk and dv
    const int32_t* cu;
    int T, n_seqs, hq, hkv, causal, tiles, q_tiles, splits;
    float scale;
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct Tile {
    int begin, len, row0;  // first row and length of the sequence; first row of the tile within it
};

// Tile number g of the sequences' tiles of BM rows, numbered sequence after sequence: one
// wave scans 64 sequences at a time. The bounds read from the device are clamped to
// [0, T] and to non-negative lengths, so that no value of theirs leads outside the
// tensors. False when there are fewer tiles. Every workgroup scans for itself, so that the scans
// grow with the square of the sequences: sequences of one token, forward and backward, us: 256 of 28/4
// heads of 64 55, 191; 1024 222, 961; 4096 3835, 8844; 16384 52 ms, 122 ms; 32768 of 4/1 29 ms, 74 ms.
// kMaxSeqs keeps the largest calls that a grid holds to seconds.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int bm, int g, Tile& t) {
    if (!a.cu) {
        t = {0, a.T, g * bm};
        return t.row0 < a.T;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
        const int s = min(s0 + lane, a.n_seqs - 1);
        const int b = min(max(a.cu[s], 0), a.T);
        const int e = min(max(a.cu[s + 1], b), a.T);
        const int n = s0 + lane < a.n_seqs ? (e - b + bm - 1) / bm : 0;
        int incl = n;
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o, 64);
            if (lane >= o) incl += v;
        }
        const int first = before + incl - n;
        const uint64_t hit = __ballot(g >= first && g < first + n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            t.begin = uni(__shfl(b, l, 64));
            t.len = uni(__shfl(e - b, l, 64));
            t.row0 = uni((g - __shfl(first, l, 64)) * bm);
            return true;
        }
        before += uni(__shfl(incl, 63, 64));
    }
    return false;
}

// The factor of dq and dk. A softmax over one key is 1 whatever its score, so nothing reaches q
// and k of a sequence of one token; what rounding leaves of dP - delta there is not passed on.
__device__ __forceinline__ float grad_scale(const AttnArgs& a, const Tile& t) { return t.len > 1 ? a.scale : 0.0f; }

// Workgroup id -> (kv head, item of that head). Items of one kv head share its K and V (or
// its queries' dO), so they are kept on as few XCDs as the head count allows: the XCD of a
// workgroup is its id mod 8, and each L2 then holds the operands of hkv / 8 heads at a time.
// False past the last item. Grids: attn_grid.
__device__ __forceinline__ bool pick_item(uint32_t b, int hkv, int items, int& head, int& item) {
    if (hkv % 8 == 0) {
        const int x = b % 8, l = b / 8;
        head = x * (hkv / 8) + l / items;
        item = l % items;
        return true;
    }
    if (8 % hkv == 0) {
        const int x = b % 8, l = b / 8, n = 8 / hkv;
        head = x / n;
        item = l * n + x % n;
        return item < items;
    }
    head = b % hkv;
    item = b / hkv;
    return true;
}

// Workgroup id for the place b of a grid that runs in one round: workgroups 256 apart share a CU,
// and with the longest first the first CU would get the longest of each 256. Every second 256
// go the other way round. Forward, heads 64 wide, us: 2048 tokens of 16/16 heads 26.3, 23.1;
// 1800: 22.8, 20.4; 4096: 62.3, 56.9; of 14/2 2048: 22.2, 22.0. Of heads 128 wide, which run two
// workgroups a CU, and in dq it gains nothing.
__device__ __forceinline__ uint32_t snake(uint32_t b, uint32_t grid) {
    const uint32_t base = b & ~255u, n = min(256u, grid - base) / 8;
    return b & 256 ? base + (n - 1 - (b - base) / 8) * 8 + b % 8 : b;  // the XCD stays
}

int64_t attn_grid(int hkv, int64_t items) {
    if (hkv % 8 != 0 && 8 % hkv == 0) return 8 * cdiv(items, 8 / hkv);
    return hkv * items;
}

// LDS image of a staged tile: rows of D bf16, the 16-byte chunk c of row r at chunk
// c ^ swz(r). LDS serves 256 bytes a cycle: 16 lanes of a 16-byte read, 32 of an 8-byte one.
// The operand read takes one chunk of 16 rows (all 16 chunks of the 256-byte line then have
// to differ: 128 / D rows share a line, swz maps the other row bits one to one), the
// transposing read two neighbouring chunk pairs of 4 rows (the rows' low bits have to move
// whole pairs of pairs).
template <int D>
__device__ __forceinline__ int swz(int r) {
    const int high = D == 128 ? (r & 3) << 2 : D == 64 ? ((r >> 1) & 1) << 2 : 0;
    return high | ((r >> 2) & 3);
}

// Per-lane byte offsets into a staged tile.
template <int D>
struct LdsMap {
    int row_chunk[D / 16];    // operand read: row l % 32, chunk 2 s + l / 32 (contraction step s)
    int tr[D / 32][2];        // transposing read: column block nb, rows 8 j + 4 (l / 32) + (l % 16) / 4
    __device__ __forceinline__ LdsMap(int lane) {
        const int r = lane & 31, h = lane >> 5, i = lane & 15, g = (lane >> 4) & 1;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) row_chunk[s] = r * 2 * D + ((2 * s + h) ^ swz<D>(r)) * 16;
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * j + 4 * h + (i >> 2);
                tr[nb][j] = row * 2 * D + ((4 * nb + 2 * g + ((i >> 1) & 1)) ^ swz<D>(row)) * 16 + (i & 1) * 8;
            }
    }
};

__device__ __forceinline__ bf16x8 lds_frag(const char* p) { return as_bf16x8(*reinterpret_cast<const u32x4*>(p)); }

// 8 contraction indices (two groups of 4 rows) of one column, from row-major LDS.
__device__ __forceinline__ bf16x8 lds_frag_tr(const char* p0, const char* p1) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p1));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return as_bf16x8(u32x4{x.x, x.y, y.x, y.y});
}

__device__ __forceinline__ bf16x8 pack8(const f32x16& v, int g) {
    return as_bf16x8(u32x4{pack_bf16x2(v[8 * g], v[8 * g + 1]), pack_bf16x2(v[8 * g + 2], v[8 * g + 3]),
                           pack_bf16x2(v[8 * g + 4], v[8 * g + 5]), pack_bf16x2(v[8 * g + 6], v[8 * g + 7])});
}

// What pack8 rounded off, rounded itself: both together hold v to 2^-16 of its size.
__device__ __forceinline__ bf16x8 pack8_rest(const f32x16& v, int g) {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = v[8 * g + 2 * e], b = v[8 * g + 2 * e + 1];
        const uint32_t x = pack_bf16x2(a, b);
        r[e] = pack_bf16x2(a - __uint_as_float(x << 16), b - __uint_as_float(x & 0xFFFF0000u));
    }
    return as_bf16x8(r);
}

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.0f;
    return z;
}

// The other half-wave's value (lane l ^ 32) combined with this lane's.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Global -> LDS copy of a tile by the W waves of the workgroup, 16 bytes a lane and
// instruction: LDS is written linearly, so the swizzle is applied to the global chunk.
template <int D, int kRows, int W>
struct TileCopy {
    static constexpr int kPieces = kRows * 2 * D / 1024;
    static constexpr int kRounds = (kPieces + W - 1) / W;
    uint32_t off[kRounds];
    // with fewer pieces than waves some are copied twice, the same bytes
    static __device__ __forceinline__ int piece(int n, int wave) { return (n * W + wave) % kPieces; }
    __device__ __forceinline__ TileCopy(int wave, int lane, int ld) {
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
            const int p = piece(n, wave) * 1024 + lane * 16;
            const int row = p / (2 * D), ch = (p / 16) % (D / 8);
            off[n] = uint32_t(row) * uint32_t(ld) * 2u + uint32_t(ch ^ swz<D>(row)) * 16u;
        }
    }
    // rows >= `rows` read as zeros
    __device__ __forceinline__ void issue(const uint16_t* base, int rows, int ld, char* lds, int wave) const {
        const auto r = make_rsrc(base, rows > 0 ? uint32_t(min(rows, kRows) - 1) * uint32_t(ld) * 2u + 2u * D : 0u);
#pragma unroll
        for (int n = 0; n < kRounds; ++n) buf_load16_lds(r, off[n], lds + piece(n, wave) * 1024);
    }
};

// Tiles [j0, j1) through two pairs of LDS buffers: tile j + 1 is copied while tile j is
// used. The four buffers have to be __shared__ variables of their own: the compiler then
// knows that a read of one does not depend on the outstanding copies to the others, and does
// not wait for them. Measured and left out: four pairs, three tiles ahead (512 tokens of 28/4
// heads 12.0 -> 14.4 us, fewer workgroups fit a CU), and the copy instructions spread between
// the first products (12.1 -> 12.5 us, more registers).
template <typename Stage, typename Compute>
__device__ __forceinline__ void double_buffered(int j0, int j1, char* a0, char* b0, char* a1, char* b1, Stage&& stage,
                                                Compute&& compute) {
    if (j0 < j1) stage(j0, a0, b0);
    auto step = [&](int j, char* a, char* b, char* a_free, char* b_free) {
        wait_vmcnt<0>();
        __syncthreads();  // every wave's share of tile j is there; the freed pair has no reader left
        if (j + 1 < j1) stage(j + 1, a_free, b_free);
        compute(j, a, b);
    };
    for (int j = j0; j < j1; j += 2) {
        step(j, a0, b0, a1, b1);
        if (j + 1 < j1) step(j + 1, a1, b1, a0, b0);
    }
}

// Where one of several waves' shares of 32 x D fp32 sums lies in the (then free) staging
// buffers, 16 bytes a lane and step. Every access strides 1 KB: lane-contiguous.
template <int D>
__device__ __forceinline__ f32x4* share_slot(int i, int buffer_bytes, char* a0, char* a1, char* b0, char* b1, int lane) {
    const int fit = buffer_bytes / (128 * D), n = i / fit;
    char* b = n == 0 ? a0 : n == 1 ? a1 : n == 2 ? b0 : b1;
    return reinterpret_cast<f32x4*>(b + i % fit * (128 * D)) + lane;
}

template <int NB>
__device__ __forceinline__ void put_share(f32x4* p, const f32x16 (&x)[NB]) {
#pragma unroll
    for (int n = 0; n < 4 * NB; ++n) {
        const int e = n % 4 * 4;
        p[64 * n] = f32x4{x[n / 4][e], x[n / 4][e + 1], x[n / 4][e + 2], x[n / 4][e + 3]};
    }
}

// x = x * f + share * g
template <int NB>
__device__ __forceinline__ void add_share(f32x16 (&x)[NB], const f32x4* p, float f, float g) {
#pragma unroll
    for (int n = 0; n < 4 * NB; ++n) {
        const f32x4 v = p[64 * n];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n / 4][n % 4 * 4 + e] = x[n / 4][n % 4 * 4 + e] * f + v[e] * g;
    }
}

// ------------------------------------------------------------------ forward

// One workgroup: R rows of waves x C waves, 32 queries of one head a row; K and V in tiles of
// 64 keys, double buffered in LDS. C = 1: a row is one wave, which takes both 32-key blocks of a
// tile. C = 2: its two waves take one block each and meet at the end. R = 2, C = 2 makes twice
// the workgroups, each half as long, for calls too small to fill the card. S^T = K Q^T puts a
// query in a lane, so the softmax statistics are one register each. The running maximum is
// raised, and o and the sum rescaled, only when some row's tile maximum exceeds it by more than
// 8 (in log2 units): p then stays below 2^8.
// Bound by the matrix and vector units in turn, at long lengths by the card's power: 8192 tokens
// of 64/8 heads of 128, causal, 1030 us, 1.07 PFLOP/s of what the mask leaves (on zeros, which
// draw less power, 758 us), without an LDS bank conflict and with 96 % of the L2 reads hits;
// 4096 in seven sequences of 40/8 heads 70 us, 610 TFLOP/s (ragged tiles); 512 tokens of 28/4
// heads 11 us: the longest row's 8 tiles one after the other.
template <int D, int R, int C>
__global__ __launch_bounds__(64 * R * C, 2) void k_attn_fwd(AttnArgs a) {
    constexpr int BM = 32 * R, B = 2 / C, kTile = 64, KS = D / 16, NB = D / 32;
    __shared__ __align__(1024) char sK0[kTile * 2 * D], sV0[kTile * 2 * D], sK1[kTile * 2 * D], sV1[kTile * 2 * D];
    const int G = a.hq / a.hkv;
    int kvh, item;
    const bool one_round = D < 128 && gridDim.x <= 1024 && gridDim.x % 8 == 0;
    if (!pick_item(one_round ? snake(blockIdx.x, gridDim.x) : blockIdx.x, a.hkv, a.tiles * G, kvh, item)) return;
    const int head = kvh * G + item % G;
    Tile t;
    if (!find_tile(a, BM, a.tiles - 1 - item / G, t)) return;  // a sequence's longest rows first
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), h = lane >> 5;
    const int wr = wave % R, wc = C == 1 ? 0 : wave / R, b0 = B * wc;  // row, place in it, first key block
    const int ldq = a.hq * D, ldk = a.hkv * D;
    const int q_lo = t.row0 + 32 * wr, q_row = q_lo + (lane & 31);
    const float c = a.scale * kLog2e;

    bf16x8 qf[KS];
    {
        const int rows = t.len - t.row0;
        const auto r = make_rsrc(a.q + (size_t(t.begin) + t.row0) * ldq + head * D,
                                 uint32_t(min(rows, BM) - 1) * uint32_t(ldq) * 2u + 2u * D);
        const uint32_t o = uint32_t(32 * wr + (lane & 31)) * uint32_t(ldq) * 2u + 16u * h;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = as_bf16x8(buf_load16(r, o + 32u * s));
    }
    const LdsMap<D> map(lane);
    const TileCopy<D, kTile, R * C> copy(wave, lane, ldk);
    const uint16_t* kb = a.k + size_t(t.begin) * ldk + kvh * D;
    const uint16_t* vb = a.v + size_t(t.begin) * ldk + kvh * D;

    f32x16 acc[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[nb] = zero16();
    // m: running maximum (-inf before the first key); base: what exponents are taken from, m
    // or 0 while there is none
    float m = -INFINITY, base = 0.0f, l = 0.0f;
    const int keys = a.causal ? min(t.len, t.row0 + BM) : t.len;
    const int n = (keys + kTile - 1) / kTile;

    auto stage = [&](int j, char* k, char* v) {
        copy.issue(kb + size_t(j) * kTile * ldk, t.len - j * kTile, ldk, k, wave);
        copy.issue(vb + size_t(j) * kTile * ldk, t.len - j * kTile, ldk, v, wave);
    };
    auto compute = [&](int j, const char* k, const char* v) {
        const int k0 = j * kTile + 32 * b0;
        if (a.causal && k0 > q_lo + 31) return;  // nothing of these keys for the wave's rows
        k += b0 * 64 * D;
        v += b0 * 64 * D;
        f32x16 s[B];
#pragma unroll
        for (int b = 0; b < B; ++b) s[b] = zero16();
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int b = 0; b < B; ++b)
                s[b] = mfma32x32x16(lds_frag(k + b * 64 * D + map.row_chunk[i]), qf[i], s[b]);
        if (k0 + 32 * B > t.len || (a.causal && k0 + 32 * B - 1 > q_lo)) {
            const int last = (a.causal ? min(q_row, t.len - 1) : t.len - 1) - k0 - 4 * h;
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (32 * b + 8 * (e / 4) + e % 4 > last) s[b][e] = -INFINITY;
        }
        float mt = s[0][0];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) mt = fmaxf(mt, s[b][e]);
        mt = max_halves(mt) * c;
        if (__any(mt > m + 8.0f)) {
            const float top = fmaxf(m, mt), to = top > -INFINITY ? top : 0.0f;
            // before the first key o and l are 0, and 2^(0 - to) may be infinite
            const float f = m > -INFINITY ? exp2f(base - to) : 0.0f;
            m = top;
            base = to;
            l *= f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[nb][e] *= f;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[b][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], c, -base));
                l += s[b][e];
            }
#pragma unroll
        for (int g = 0; g < 2 * B; ++g) {
            const bf16x8 p = pack8(s[g / 2], g % 2);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                acc[nb] = mfma32x32x16(lds_frag_tr(v + g * 32 * D + map.tr[nb][0], v + g * 32 * D + map.tr[nb][1]), p,
                                       acc[nb]);
        }
    };
    double_buffered(0, n, sK0, sV0, sK1, sV1, stage, compute);
    l = sum_halves(l);
    if constexpr (C > 1) {  // the waves of a row hand their shares to its first
        __shared__ float sML[R * C][2][64];  // the exponents' base and the sum; no share without a key
        __syncthreads();
        if (wc > 0) {
            put_share(share_slot<D>((wc - 1) * R + wr, sizeof sK0, sK0, sV0, sK1, sV1, lane), acc);
            sML[wave][0][lane] = m > -INFINITY ? base : -INFINITY;
            sML[wave][1][lane] = l;
        }
        __syncthreads();
        if (wc > 0) return;
#pragma unroll
        for (int i = 1; i < C; ++i) {
            const float other = sML[i * R + wr][0][lane];
            const float to = fmaxf(base, other);  // the first wave has seen key 0: finite
            const float f0 = exp2f(base - to), f1 = exp2f(other - to);
            base = to;
            l = l * f0 + sML[i * R + wr][1][lane] * f1;
            add_share(acc, share_slot<D>((i - 1) * R + wr, sizeof sK0, sK0, sV0, sK1, sV1, lane), f0, f1);
        }
    }
    if (q_row < t.len) {
        const size_t row = size_t(t.begin) + q_row;
        const float inv = 1.0f / l;
        uint16_t* out = a.out + row * ldq + head * D;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<u32x2*>(out + 32 * nb + 2 * e + 4 * h) =
                    u32x2{pack_bf16x2(acc[nb][e] * inv, acc[nb][e + 1] * inv),
                          pack_bf16x2(acc[nb][e + 2] * inv, acc[nb][e + 3] * inv)};
        if (h == 0) a.lse[size_t(head) * a.T + row] = (base + log2f(l)) * kLn2;
    }
}

// ------------------------------------------------------------------ backward: dq (and delta)

// As the forward, with dO beside Q in registers: per 64-key tile S^T = K Q^T,
// dP^T = V dO^T, dS^T in place, dq^T += K^T dS^T. delta is formed here first (the dk/dv
// kernel behind this one reads it). R, C and B as in the forward. FINE: for calls of at
// most 64 rows, and for heads 32 wide, whose rounding grows with the length instead (dq 1.49 times
// its own at 512 rows, 64 and 128 wide 1.44). Measured (us, one bf16 value for dS and two):
// 4096 tokens of 4/1 heads of 32 48.1, 59.0; 64 tokens of 64/8 heads of 128 15.4, 15.6.
// Bound as the forward: 8192 tokens of 64/8 heads of 128 1364 us, 1.21 PFLOP/s with its share
// (S, dP and dq: 6 D operations a pair).
template <int D, int R, int C, bool STATS, bool FINE>
__device__ __forceinline__ void bwd_dq(const AttnArgs& a, uint32_t block, char* sK0, char* sV0, char* sK1, char* sV1) {
    constexpr int BM = 32 * R, B = 2 / C, kTile = 64, KS = D / 16, NB = D / 32;
    const int G = a.hq / a.hkv;
    int kvh, item;
    if (!pick_item(block, a.hkv, a.q_tiles * G, kvh, item)) return;
    const int head = kvh * G + item % G;
    Tile t;
    if (!find_tile(a, BM, a.q_tiles - 1 - item / G, t)) return;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), h = lane >> 5;
    const int wr = wave % R, wc = C == 1 ? 0 : wave / R, b0 = B * wc;
    const int ldq = a.hq * D, ldk = a.hkv * D;
    const int q_lo = t.row0 + 32 * wr, q_row = q_lo + (lane & 31);
    const float c = a.scale * kLog2e;

    const TileCopy<D, kTile, R * C> copy(wave, lane, ldk);
    const uint16_t* kb = a.k + size_t(t.begin) * ldk + kvh * D;
    const uint16_t* vb = a.v + size_t(t.begin) * ldk + kvh * D;
    auto stage = [&](int j, char* k, char* v) {
        copy.issue(kb + size_t(j) * kTile * ldk, t.len - j * kTile, ldk, k, wave);
        copy.issue(vb + size_t(j) * kTile * ldk, t.len - j * kTile, ldk, v, wave);
    };

    bf16x8 qf[KS], df[KS];
    float delta = 0.0f;
    {
        const int rows = t.len - t.row0;
        const size_t at = (size_t(t.begin) + t.row0) * ldq + head * D;
        const uint32_t bytes = uint32_t(min(rows, BM) - 1) * uint32_t(ldq) * 2u + 2u * D;
        const auto rq = make_rsrc(a.q + at, bytes), rd = make_rsrc(a.dO + at, bytes), ro = make_rsrc(a.o + at, bytes);
        const uint32_t o = uint32_t(32 * wr + (lane & 31)) * uint32_t(ldq) * 2u + 16u * h;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s] = as_bf16x8(buf_load16(rq, o + 32u * s));
            df[s] = as_bf16x8(buf_load16(rd, o + 32u * s));
            const bf16x8 of = as_bf16x8(buf_load16(ro, o + 32u * s));
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(float(df[s][e]), float(of[e]), delta);
        }
        delta = sum_halves(delta);
    }
    float lse2 = 0.0f;
    if (q_row < t.len) {
        const size_t at = size_t(head) * a.T + t.begin + q_row;
        lse2 = a.lse_in[at] * kLog2e;
        if (STATS && h == 0 && wc == 0) {
            a.stats[at] = lse2;
            a.stats[size_t(a.hq) * a.T + at] = delta;
        }
    }
    const LdsMap<D> map(lane);

    f32x16 acc[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[nb] = zero16();
    const int keys = a.causal ? min(t.len, t.row0 + BM) : t.len;
    const int n = (keys + kTile - 1) / kTile;
    auto compute = [&](int j, const char* k, const char* v) {
        const int k0 = j * kTile + 32 * b0;
        if (a.causal && k0 > q_lo + 31) return;
        k += b0 * 64 * D;
        v += b0 * 64 * D;
        const bool edge = k0 + 32 * B > t.len || (a.causal && k0 + 32 * B - 1 > q_lo);
        const int last = (a.causal ? min(q_row, t.len - 1) : t.len - 1) - k0 - 4 * h;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            f32x16 s = zero16(), dp;
#pragma unroll
            for (int e = 0; e < 16; ++e) dp[e] = -delta;  // dP - delta straight from the accumulator
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                s = mfma32x32x16(lds_frag(k + b * 64 * D + map.row_chunk[i]), qf[i], s);
                dp = mfma32x32x16(lds_frag(v + b * 64 * D + map.row_chunk[i]), df[i], dp);
            }
            if (edge) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (32 * b + 8 * (e / 4) + e % 4 > last) s[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -lse2)) * dp[e];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const bf16x8 ds = pack8(s, g);
                const char* kg = k + (2 * b + g) * 32 * D;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const bf16x8 kt = lds_frag_tr(kg + map.tr[nb][0], kg + map.tr[nb][1]);
                    acc[nb] = mfma32x32x16(kt, ds, acc[nb]);
                    if constexpr (FINE) acc[nb] = mfma32x32x16(kt, pack8_rest(s, g), acc[nb]);
                }
            }
        }
    };
    double_buffered(0, n, sK0, sV0, sK1, sV1, stage, compute);
    if constexpr (C > 1) {  // the waves of a row hand their shares to its first
        __syncthreads();
        if (wc > 0) put_share(share_slot<D>((wc - 1) * R + wr, kTile * 2 * D, sK0, sV0, sK1, sV1, lane), acc);
        __syncthreads();
        if (wc > 0) return;
#pragma unroll
        for (int i = 1; i < C; ++i)
            add_share(acc, share_slot<D>((i - 1) * R + wr, kTile * 2 * D, sK0, sV0, sK1, sV1, lane), 1.0f, 1.0f);
    }
    if (q_row < t.len) {
        uint16_t* out = a.dq + (size_t(t.begin) + q_row) * ldq + head * D;
        const float f = grad_scale(a, t);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<u32x2*>(out + 32 * nb + 2 * e + 4 * h) =
                    u32x2{pack_bf16x2(acc[nb][e] * f, acc[nb][e + 1] * f),
                          pack_bf16x2(acc[nb][e + 2] * f, acc[nb][e + 3] * f)};
    }
}

template <int D, int R, int C>
__global__ __launch_bounds__(64 * R * C, 2) void k_attn_bwd_dq(AttnArgs a) {
    __shared__ __align__(1024) char sK0[128 * D], sV0[128 * D], sK1[128 * D], sV1[128 * D];
    bwd_dq<D, R, C, true, D == 32>(a, blockIdx.x, sK0, sV0, sK1, sV1);
}

// ------------------------------------------------------------------ backward: dk, dv

// Where a workgroup's share of dk and dv begins in the workspace, in 16-byte units.
template <int D>
__device__ __forceinline__ size_t share_of(int tile, int kvh, int split, const AttnArgs& a) {
    return ((size_t(tile) * a.hkv + kvh) * a.splits + split) * (2 * kKeyWaves * 8 * D);
}

// One workgroup: 8 waves, KW blocks of 32 keys of one kv head x QW. K and V stay in LDS; the
// queries of the G heads pass through LDS in tiles of 32 QW (Q, dO, lse, delta), 32 to each of
// the QW waves of a key block, whose sums meet at the end. Per 32 queries S = Q K^T,
// dP = dO V^T (a key in a lane), dv^T += dO^T P, dk^T += Q^T dS.
// With splits > 1 the (head, query tile) list is cut into contiguous ranges, one a
// workgroup, whose fp32 shares k_attn_bwd_join adds in order.
// Bound by LDS reads beside the products (every operand of S and dP is read anew, Q and dO once
// more transposed) and at long lengths by power: 8192 tokens of 64/8 heads of 128 2070 us,
// 1.06 PFLOP/s (S, dP, dv and dk: 8 D operations a pair). K and V in registers leave room for
// one wave a SIMD only (the whole backward 4027 us at those sizes, against 3497 with V in LDS);
// K alone there leaves none for fragments read ahead (1024 tokens of 28/4 heads of 128 61.2 ->
// 57.5 us with K in LDS too, 512 of 64/8 51.0 -> 48.5). Measured and left out: the products
// ordered by hand (slower); a higher wave priority around them, or for one of the two waves of a
// SIMD (no change); the second wave of a key block half a tile behind the first, whose third
// pair of buffers and state do not fit beside K (with K in registers five times slower at width
// 128, 15 % at 64).
// LDS of a dk/dv workgroup: K; V; two pairs of a tile's Q, and its dO with the rows' lse * log2 e
// and delta behind it.
template <int D>
struct DkvLds {
    static constexpr int QW = 2, BQ = 32 * QW, QB = BQ * 2 * D, SB = 256, DB = QB + 2 * SB, KB = 64 * kKeyWaves * D;
};

template <int D, bool FINE>
__device__ __forceinline__ void bwd_dkv(const AttnArgs& a, uint32_t block, char* sK, char* sV, char* sQ0, char* sD0,
                                        char* sQ1, char* sD1) {
    using L = DkvLds<D>;
    constexpr int KW = kKeyWaves, QW = L::QW, W = KW * QW, BM = 32 * KW, KS = D / 16, NB = D / 32, BQ = L::BQ;
    constexpr int QB = L::QB, SB = L::SB;
    const int G = a.hq / a.hkv;
    int kvh, item;
    if (!pick_item(block, a.hkv, a.tiles * a.splits, kvh, item)) return;
    const int split = item % a.splits;
    Tile t;
    const int tile = item / a.splits;
    if (!find_tile(a, BM, tile, t)) return;  // causal: the first keys have the most queries
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), h = lane >> 5;
    const int ldq = a.hq * D, ldk = a.hkv * D;
    const int kw = wave % KW, qw = wave / KW;
    const int k_lo = t.row0 + 32 * kw, key = k_lo + (lane & 31);
    const float c = a.scale * kLog2e;

    // (query tile, head) pairs: the tiles from the last down to the first that sees a key of
    // this workgroup, and the heads of each. The workgroups of a kv head run side by side on
    // one XCD: in this order all of them want the same Q and dO at about the same time, and
    // find them in its L2.
    const int tile_lo = a.causal ? t.row0 / BQ : 0, tile_hi = (t.len - 1) / BQ;
    const int total = G * (tile_hi + 1 - tile_lo);
    const int i0 = int(int64_t(split) * total / a.splits), i1 = int(int64_t(split + 1) * total / a.splits);

    {
        const size_t at = (size_t(t.begin) + t.row0) * ldk + kvh * D;
        const int rows = min(t.len - t.row0, BM);
        const TileCopy<D, BM, W> keys(wave, lane, ldk);
        keys.issue(a.k + at, rows, ldk, sK, wave);
        keys.issue(a.v + at, rows, ldk, sV, wave);
    }
    const LdsMap<D> map(lane);
    const TileCopy<D, BQ, W> copy(wave, lane, ldq);
    int next = tile_hi - i0 / G, g_next = i0 % G;  // of the tile to be staged
    auto stage = [&](int, char* q, char* d) {
        const int q0 = next * BQ, head = kvh * G + g_next, rows = t.len - q0;
        const size_t at = (size_t(t.begin) + q0) * ldq + head * D;
        copy.issue(a.q + at, rows, ldq, q, wave);
        copy.issue(a.dO + at, rows, ldq, d, wave);
        // rows past the sequence read as zeros, like their q and dO: P = 1 then multiplies zeros only
        if (wave < 2 * SB / 256) {
            constexpr int per = SB / 256;  // waves for each of lse and delta
            const int x = wave / per, r0 = wave % per * 64;
            const auto r = make_rsrc(a.stats + (size_t(x) * a.hq + head) * a.T + t.begin + q0,
                                     uint32_t(min(rows, BQ)) * 4u);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(d + QB + wave * 256), 4, (r0 + lane) * 4, 0, 0, 0);
        }
        if (++g_next == G) g_next = 0, --next;
    };

    f32x16 dk[NB], dv[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) dk[nb] = zero16(), dv[nb] = zero16();
    int cur = tile_hi - i0 / G, g_cur = i0 % G;
    auto compute = [&](int, const char* q, const char* d) {
        const int q0 = cur * BQ + 32 * qw;
        if (++g_cur == G) g_cur = 0, --cur;
        if (a.causal && q0 + 31 < k_lo) return;  // all the wave's queries come before its keys
        const f32x4* stat = reinterpret_cast<const f32x4*>(d + QB + 128 * qw) + h;
        q += qw * 64 * D;
        d += qw * 64 * D;
        f32x16 s = zero16(), dp;
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[e] = -stat[SB / 16 + e / 4 * 2][e % 4];  // dP - delta straight from the accumulator
        const char *v = sV + kw * 64 * D, *k = sK + kw * 64 * D;
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            s = mfma32x32x16(lds_frag(q + map.row_chunk[e]), lds_frag(k + map.row_chunk[e]), s);
            dp = mfma32x32x16(lds_frag(d + map.row_chunk[e]), lds_frag(v + map.row_chunk[e]), dp);
        }
        if (a.causal && q0 < k_lo + 31) {
            const int first = key - q0 - 4 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * (e / 4) + e % 4 < first) s[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -stat[e / 4 * 2][e % 4]));
            dp[e] *= s[e];
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const bf16x8 p = pack8(s, g), ds = pack8(dp, g);
            const char *dg = d + g * 32 * D, *qg = q + g * 32 * D;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                dv[nb] = mfma32x32x16(lds_frag_tr(dg + map.tr[nb][0], dg + map.tr[nb][1]), p, dv[nb]);
                const bf16x8 qt = lds_frag_tr(qg + map.tr[nb][0], qg + map.tr[nb][1]);
                dk[nb] = mfma32x32x16(qt, ds, dk[nb]);
                if constexpr (FINE) dk[nb] = mfma32x32x16(qt, pack8_rest(dp, g), dk[nb]);
            }
        }
    };
    double_buffered(i0, i1, sQ0, sD0, sQ1, sD1, stage, compute);
    wait_vmcnt<0>();  // without a tile to use them, the copies of K and V are still under way
    // The sums of a key block: its second wave hands them to the first through the staging
    // buffers, dk first, then dv.
    auto meet = [&](f32x16(&x)[NB]) {
        __syncthreads();
        if (qw > 0) put_share(share_slot<D>(kw, QB, sQ0, sQ1, sD0, sD1, lane), x);
        __syncthreads();
        if (qw == 0) add_share(x, share_slot<D>(kw, QB, sQ0, sQ1, sD0, sD1, lane), 1.0f, 1.0f);
    };
    meet(dk);
    meet(dv);
    if (qw > 0) return;
    if (a.splits == 1) {
        if (key >= t.len) return;
        const size_t at = (size_t(t.begin) + key) * ldk + kvh * D + 4 * h;
        const float f = grad_scale(a, t);
#pragma unroll
        for (int n = 0; n < 4 * NB; ++n) {
            const int nb = n / 4, e = n % 4 * 4;
            *reinterpret_cast<u32x2*>(a.dk + at + 8 * n) =
                u32x2{pack_bf16x2(dk[nb][e] * f, dk[nb][e + 1] * f), pack_bf16x2(dk[nb][e + 2] * f, dk[nb][e + 3] * f)};
            *reinterpret_cast<u32x2*>(a.dv + at + 8 * n) =
                u32x2{pack_bf16x2(dv[nb][e], dv[nb][e + 1]), pack_bf16x2(dv[nb][e + 2], dv[nb][e + 3])};
        }
        return;
    }
    // a share as the lanes hold it, whole kilobytes a store
    f32x4* part = reinterpret_cast<f32x4*>(a.part) + share_of<D>(tile, kvh, split, a) + kw * 256 * NB + lane;
#pragma unroll
    for (int n = 0; n < 4 * NB; ++n) {
        const int nb = n / 4, e = n % 4 * 4;
        part[64 * n] = f32x4{dk[nb][e], dk[nb][e + 1], dk[nb][e + 2], dk[nb][e + 3]};
        part[64 * n + KW * 256 * NB] = f32x4{dv[nb][e], dv[nb][e + 1], dv[nb][e + 2], dv[nb][e + 3]};
    }
}

template <int D>
__global__ __launch_bounds__(512, 2) void k_attn_bwd_dkv(AttnArgs a) {
    using L = DkvLds<D>;
    __shared__ __align__(1024) char sK[L::KB], sV[L::KB], sQ0[L::QB], sD0[L::DB], sQ1[L::QB], sD1[L::DB];
    bwd_dkv<D, false>(a, blockIdx.x, sK, sV, sQ0, sD0, sQ1, sD1);
}

// Both in one launch, for calls whose dq and dk/dv workgroups would each leave the card partly
// idle: the first q_wgs workgroups take 128 rows of dq each, with two waves a row. lse * log2 e
// and delta come from k_attn_bwd_stats, since neither kind can wait for the other. FINE: calls
// of at most 64 tokens that k_attn_bwd_few does not take. 512 tokens of 28/4 heads of 128: 24 us,
// with the row statistics before and the join behind of 4 us each; 2048 tokens of 16/16 heads of
// 64 in three sequences without a mask 58 us, 400 TFLOP/s.
template <int D, bool FINE>
__global__ __launch_bounds__(512, 2) void k_attn_bwd_both(AttnArgs a, uint32_t q_wgs) {
    using L = DkvLds<D>;
    __shared__ __align__(1024) char sK[L::KB], sV[L::KB], sQ0[L::QB], sD0[L::DB], sQ1[L::QB], sD1[L::DB];
    if (blockIdx.x < q_wgs)
        bwd_dq<D, 4, 2, false, FINE || D == 32>(a, blockIdx.x, sQ0, sD0, sQ1, sD1);
    else
        bwd_dkv<D, FINE>(a, blockIdx.x - q_wgs, sK, sV, sQ0, sD0, sQ1, sD1);
}

// dk and dv of a call of few tokens: 32 keys of one kv head a workgroup, and each of its 8 waves
// 32 queries of a head at a time, with a part of LDS and row statistics of its own, so that the
// G heads of a kv head are taken side by side; the waves' sums meet at the end, in wave order.
// As bwd_dkv with FINE otherwise. Bound by latency, of one load, one tile and two sums through
// LDS: 2 tokens of 28/4 heads of 128 9.8 us with the launch.
template <int D>
struct FewLds {
    static constexpr int W = 8, BB = 64 * D, SUM = 128 * D;  // bytes of 32 rows; of a wave's sums of dk or dv
    static constexpr int ALL = W * 2 * BB;                   // every wave's Q and dO; then every wave's sums
};

template <int D>
__device__ __forceinline__ void bwd_dkv_few(const AttnArgs& a, uint32_t block, char* sK, char* sV, char* sB, float* sStat) {
    using L = FewLds<D>;
    constexpr int W = L::W, KS = D / 16, NB = D / 32;
    static_assert(L::ALL == W * L::SUM, "the sums take the place of Q and dO");
    const int G = a.hq / a.hkv;
    int kvh, tile;
    if (!pick_item(block, a.hkv, a.tiles, kvh, tile)) return;
    Tile t;
    if (!find_tile(a, 32, tile, t)) return;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), h = lane >> 5;
    const int ldq = a.hq * D, ldk = a.hkv * D;
    const float c = a.scale * kLog2e;
    {
        const size_t at = (size_t(t.begin) + t.row0) * ldk + kvh * D;
        const TileCopy<D, 32, W> keys(wave, lane, ldk);
        keys.issue(a.k + at, t.len - t.row0, ldk, sK, wave);
        keys.issue(a.v + at, t.len - t.row0, ldk, sV, wave);
    }
    const LdsMap<D> map(lane);
    const TileCopy<D, 32, 1> copy(0, lane, ldq);
    char *q = sB + wave * 2 * L::BB, *d = q + L::BB;
    float* stat = sStat + wave * 64;

    f32x16 dk[NB], dv[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) dk[nb] = zero16(), dv[nb] = zero16();
    const int first_q = a.causal ? t.row0 / 32 : 0, nq = (t.len - 1) / 32 + 1 - first_q;  // a head's blocks that see a key
    const int total = G * nq;
    for (int i0 = 0; i0 < total; i0 += W) {
        const int i = i0 + wave, q0 = (first_q + i % nq) * 32;
        if (i0 > 0) __syncthreads();  // the last round's reads are done
        if (i < total) {
            const int head = kvh * G + i / nq, rows = t.len - q0, row = lane & 31;
            const size_t at = (size_t(t.begin) + q0) * ldq + head * D;
            copy.issue(a.q + at, rows, ldq, q, 0);
            copy.issue(a.dO + at, rows, ldq, d, 0);
            const uint32_t bytes = uint32_t(min(rows, 32) - 1) * uint32_t(ldq) * 2u + 2u * D;
            const auto rd = make_rsrc(a.dO + at, bytes), ro = make_rsrc(a.o + at, bytes);
            const uint32_t o = uint32_t(row) * uint32_t(ldq) * 2u + 16u * h;
            float delta = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf16x8 df = as_bf16x8(buf_load16(rd, o + 32u * s)), of = as_bf16x8(buf_load16(ro, o + 32u * s));
#pragma unroll
                for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(float(df[e]), float(of[e]), delta);
            }
            delta = sum_halves(delta);
            if (h == 0) {
                stat[row] = row < rows ? a.lse_in[size_t(head) * a.T + t.begin + q0 + row] * kLog2e : 0.0f;
                stat[32 + row] = delta;
            }
        }
        wait_vmcnt<0>();
        __syncthreads();
        if (i >= total) continue;
        const f32x4* st = reinterpret_cast<const f32x4*>(stat) + h;
        f32x16 s = zero16(), dp;
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[e] = -st[8 + e / 4 * 2][e % 4];
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            s = mfma32x32x16(lds_frag(q + map.row_chunk[e]), lds_frag(sK + map.row_chunk[e]), s);
            dp = mfma32x32x16(lds_frag(d + map.row_chunk[e]), lds_frag(sV + map.row_chunk[e]), dp);
        }
        if (a.causal && q0 < t.row0 + 31) {
            const int first = t.row0 + (lane & 31) - q0 - 4 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * (e / 4) + e % 4 < first) s[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -st[e / 4 * 2][e % 4]));
            dp[e] *= s[e];
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const bf16x8 p = pack8(s, g), ds = pack8(dp, g), rest = pack8_rest(dp, g);
            const char *dg = d + g * 32 * D, *qg = q + g * 32 * D;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                dv[nb] = mfma32x32x16(lds_frag_tr(dg + map.tr[nb][0], dg + map.tr[nb][1]), p, dv[nb]);
                const bf16x8 qt = lds_frag_tr(qg + map.tr[nb][0], qg + map.tr[nb][1]);
                dk[nb] = mfma32x32x16(qt, ds, dk[nb]);
                dk[nb] = mfma32x32x16(qt, rest, dk[nb]);
            }
        }
    }
    const int n_sums = min(total, W);
    auto meet = [&](const f32x16(&x)[NB], uint16_t* out, float f) {
        __syncthreads();
        if (wave < n_sums) put_share(reinterpret_cast<f32x4*>(sB + wave * L::SUM) + lane, x);
        __syncthreads();
        for (int n = wave; n < 4 * NB; n += W) {
            const f32x4* p = reinterpret_cast<const f32x4*>(sB) + 64 * n + lane;
            f32x4 sum = p[0];
            for (int w = 1; w < n_sums; ++w) sum += p[w * (L::SUM / 16)];
            const int key = t.row0 + (lane & 31);
            if (key < t.len)
                *reinterpret_cast<u32x2*>(out + (size_t(t.begin) + key) * ldk + kvh * D + 8 * n + 4 * h) =
                    u32x2{pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f)};
        }
    };
    meet(dk, a.dk, grad_scale(a, t));
    meet(dv, a.dv, 1.0f);
}

// The whole backward of a call of few tokens in one launch.
template <int D>
__global__ __launch_bounds__(512, 2) void k_attn_bwd_few(AttnArgs a, uint32_t q_wgs) {
    using L = FewLds<D>;
    __shared__ __align__(1024) char sB[L::ALL], sK[L::BB], sV[L::BB];
    __shared__ __align__(16) float sStat[L::W * 64];
    if (blockIdx.x < q_wgs)
        bwd_dq<D, 4, 2, false, true>(a, blockIdx.x, sB, sB + 128 * D, sB + 256 * D, sB + 384 * D);
    else
        bwd_dkv_few<D>(a, blockIdx.x - q_wgs, sK, sV, sB, sStat);
}

// stats[0] = lse * log2 e, stats[1] = delta = do . o for every row and head: D / 8 lanes each.
// Memory bound; at the sizes that take it (7.3 MB at 512 tokens of 28/4 heads) a launch's own
// 4 us.
template <int D>
__global__ __launch_bounds__(256) void k_attn_bwd_stats(AttnArgs a) {
    constexpr int LN = D / 8;
    const int64_t n = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LN, all = int64_t(a.T) * a.hq;
    if (n >= all) return;  // whole groups of LN lanes
    const int head = int(n % a.hq), x = threadIdx.x % LN;
    const int64_t row = n / a.hq;
    const bf16x8 d = as_bf16x8(*reinterpret_cast<const u32x4*>(a.dO + n * D + 8 * x));
    const bf16x8 o = as_bf16x8(*reinterpret_cast<const u32x4*>(a.o + n * D + 8 * x));
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(float(d[e]), float(o[e]), s);
#pragma unroll
    for (int m = 1; m < LN; m *= 2) s += __shfl_xor(s, m, 64);
    if (x == 0) {
        const size_t at = size_t(head) * a.T + row;
        a.stats[at] = a.lse_in[at] * kLog2e;
        a.stats[size_t(a.hq) * a.T + at] = s;
    }
}

// dk = RNbf(scale * sum of the shares), dv = RNbf(sum of the shares), in split order; four
// of a lane's elements a thread, 2 KW NB workgroups a tile and kv head. 8 shares of 512 tokens
// and 4 heads of 128 (16.8 MB) take 4 us.
template <int D>
__global__ __launch_bounds__(256) void k_attn_bwd_join(AttnArgs a) {
    constexpr int KW = kKeyWaves, NB = D / 32;
    const int i = blockIdx.x % (2 * KW * NB), th = blockIdx.x / (2 * KW * NB);
    const int is_dv = i / (KW * NB), kw = i / NB % KW, nb = i % NB;
    const int tile = th / a.hkv, kvh = th % a.hkv, lane = threadIdx.x & 63, n = 4 * nb + (threadIdx.x >> 6);
    Tile t;
    if (!find_tile(a, 32 * KW, tile, t)) return;
    const int key = t.row0 + 32 * kw + (lane & 31);
    if (key >= t.len) return;
    const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + share_of<D>(tile, kvh, 0, a) +
                     (is_dv * KW + kw) * 256 * NB + 64 * n + lane;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) s += p[size_t(z) * (2 * KW * 256 * NB)];
    const float f = is_dv ? 1.0f : grad_scale(a, t);
    const size_t at = (size_t(t.begin) + key) * (a.hkv * D) + kvh * D + 8 * n + 4 * (lane >> 5);
    *reinterpret_cast<u32x2*>((is_dv ? a.dv : a.dk) + at) =
        u32x2{pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f)};
}

int64_t tiles_of(int64_t T, const void* cu, int64_t n_seqs, int bm) {
    return cu ? T / bm + n_seqs : cdiv(T, bm);
}

// Whether tiles of 128 rows would not even give every CU its resident workgroups (2, 3 or 4
// of head width 128, 64, 32) once; the forward then takes 64 rows a workgroup. Us with 128 and
// 64 rows: 512 tokens of 28/4 heads of 128 14.8, 12.2; 1024: 24.4, 21.0; 2048: 49.1, 50.0;
// 2048 tokens of 40/8: 55.4, 64.3; 4096 tokens of 14/2 heads of 64: 57.4, 46.7.
bool few_rows(int64_t T, int64_t hq, int64_t D) { return cdiv(T, 128) * hq < 256 * (D == 128 ? 2 : D == 64 ? 3 : 4); }

// Calls whose dk has dS as two bf16 values (dq: those, and all heads 32 wide). By all rows of the
// call, since the scatter of few results is what it bounds.
bool fine_ds(int64_t T) { return T <= 64; }

// Those of them whose dk and dv take a kv head's queries side by side (bwd_dkv_few) instead of
// one after the other: where a sequence's blocks of 32 queries of all G heads keep 8 waves busy
// once. Us one after the other and side by side: 32 tokens of 28/4 heads of 128 15.3, 11.9, of 64/8
// 15.3, 12.7; three times 20 tokens of 64/8 24.3, 13.1; 40 of 4/1 heads of 32 10.1, 5.9; with
// two rounds of blocks 64 tokens of 64/8 15.6, 19.4.
bool few_tokens(int64_t T, int64_t n_seqs, int64_t hq, int64_t hkv) {
    return fine_ds(T) && hq / hkv * cdiv(T, std::max<int64_t>(1, n_seqs) * 32) <= 8;
}

// Whether the backward takes both kinds of workgroups in one launch: up to one and a half
// workgroups of dq a CU. Us in two launches and in one: 512 tokens of 28/4 heads 39.8, 32.5;
// 1024: 68.7, 60.8; 2048: 150.7, 164.7; 1408 tokens of 32/32 heads of 64: 92.1, 85.6; 4096 of
// 14/2: 142.9, 148.1.
bool one_launch(int64_t T, int64_t hq) { return fine_ds(T) || cdiv(T, 128) * hq <= 384; }

// Shares of dk and dv: the power of two up to 16 that is expected to take the least time. A CU
// holds one workgroup of 8 waves, so the workgroups of a launch (with those of dq, where they
// share it) run in rounds of 256. A tile of 64 queries takes about 1.9 us (head width 128),
// one of 64 keys in dq half that, starting and ending a workgroup 5 us, or 8 when it stores a
// share; the shares are written and read again, in a launch of 4 us more, at about 6 TB/s, or
// 9 while the caches hold them all. Under a causal mask, and among sequences of different
// lengths, the longest workgroup has about twice the average's tiles. Measured (us, whole
// backward): 8192 tokens of 64/8 heads 3545 with one share, 3618 with 2; 4096: 1170 with 1, 932
// with 2; 512 of 28/4: 40.6, 32.3 and 38.0 with 4, 8 and 16; 1408 of 8/8, no mask: 51.6 and
// 65.0 with 1 and 2; 1408 of 4/4 heads of 64: 31.7, 29.0 and 32.7 with 1, 2 and 4; no
// share has fewer than 1.7 tiles: 64 of 28/4 19.0 and 15.3 with 1 and 4 (1.75 tiles), 100 of 64/8
// 18.7 and 20.9 with 4 and 8.
int pick_splits(int64_t T, int64_t n_seqs, int hq, int hkv, int D, int causal) {
    const int64_t seqs = std::max<int64_t>(1, n_seqs);
    const double wgs = double(std::max(cdiv(T, 32 * kKeyWaves), seqs) * hkv);
    const double dq_wgs = one_launch(T, hq) ? double(std::max(cdiv(T, 128), seqs) * hq) : 0.0;
    const int64_t len = cdiv(T, seqs * 64);                    // tiles of an average sequence
    const double avg = causal ? (len + 1) * 0.5 : double(len);  // that an average row or key meets
    const double tiles = double(hq / hkv) * avg, tile_us = 1.9 * D / 128;
    const double dq_us = 0.5 * tile_us * avg + 5, share_bytes = wgs * (2 * 32 * kKeyWaves * D * 4);
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 16 && (s == 1 || tiles >= 1.7 * s); s *= 2) {
        const double ends_us = s == 1 ? 3 + 2.0 * D / 128 : 4 + 4.0 * D / 128;
        const double run = tiles / s * tile_us, one = run + ends_us, bytes = s * share_bytes;
        const double all = wgs * s + dq_wgs, rounds = std::ceil(all / 256);
        double us;
        if (causal || seqs > 1)  // many rounds even out, a few go by the average
            us = std::max(one + run, rounds < 5 ? rounds * (wgs * s * one + dq_wgs * dq_us) / all
                                                : (wgs * s * one + dq_wgs * dq_us) / 256 + run / 6);
        else
            us = rounds * std::max(one, dq_wgs > 0 ? dq_us : 0.0);
        if (s > 1) us += 4 + 2 * bytes / (bytes < 128e6 ? 9e6 : 6e6);
        if (s == 1 || us < 0.99 * least) best = s, least = us;
    }
    return best;
}

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

int check_attn(const char* fn, int64_t T, int64_t hq, int64_t hkv, int64_t D, const int32_t* cu, int64_t n_seqs,
               int causal, float scale) {
    if (D != 32 && D != 64 && D != 128)
        return fail(NF4_E_SHAPE, "%s: head_dim must be 32, 64 or 128 (got %lld)", fn, (long long)D);
    if (T < 0 || T > (int64_t(1) << 23) || hkv <= 0 || hq <= 0 || hq % hkv != 0 || hq > 1024)
        return fail(NF4_E_SHAPE, "%s: need 0 <= T <= 2^23 and hkv | hq <= 1024 (got T=%lld hq=%lld hkv=%lld)", fn,
                    (long long)T, (long long)hq, (long long)hkv);
    if (cu ? (n_seqs < 1 || n_seqs > kMaxSeqs) : (n_seqs != 0 && n_seqs != 1))
        return fail(NF4_E_SHAPE, "%s: need 1 <= n_seqs <= 2^16 with cu_seqlens, 0 or 1 without (got %lld)", fn,
                    (long long)n_seqs);
    if (causal != 0 && causal != 1) return fail(NF4_E_ARG, "%s: causal must be 0 or 1 (got %d)", fn, causal);
    if (!std::isfinite(scale) || scale <= 0.0f)
        return fail(NF4_E_ARG, "%s: scale must be finite and positive (got %g)", fn, double(scale));
    if (cu && reinterpret_cast<uintptr_t>(cu) % 4 != 0)
        return fail(NF4_E_ARG, "%s: cu_seqlens must be 4-byte aligned", fn);
    return NF4_OK;
}

// The first n_out ranges are written: none of them may meet another range of the list.
int check_apart(const char* fn, const ByteRange* r, int n_out, int n) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (r[i].meets(r[j])) return fail(NF4_E_ARG, "%s: an output overlaps another argument", fn);
    return NF4_OK;
}

struct AttnBwdPlan {
    int splits;
    size_t stats_bytes, part_bytes;
};

AttnBwdPlan plan_bwd_attn(int64_t T, int64_t hq, int64_t hkv, int64_t D, int64_t n_seqs, int causal) {
    AttnBwdPlan p{};
    const size_t tiles = size_t(T) / (32 * kKeyWaves) + std::max<int64_t>(1, n_seqs);
    p.splits = few_tokens(T, n_seqs, hq, hkv) ? 1 : pick_splits(T, n_seqs, int(hq), int(hkv), int(D), causal);
    p.stats_bytes = (size_t(T) * hq * 8 + 255) & ~size_t(255);
    p.part_bytes = p.splits > 1 ? size_t(2) * p.splits * tiles * 32 * kKeyWaves * hkv * D * 4 : 0;
    return p;
}

// Whether a launch's threads pass the 32 bits of a grid: refused.
int check_grid(const char* fn, int64_t wgs, int threads) {
    if (wgs * threads > 0xFFFFFFFFll) return fail(NF4_E_SHAPE, "%s: too many tiles (%lld workgroups)", fn, (long long)wgs);
    return NF4_OK;
}

// Waves of a row in calls that fill the card (forward and dq): two for heads 64 wide, whose tiles
// are too short for one wave to hide their loads, one for the others. Us with one and two: 64
// wide, 8192 tokens of 16/16 heads 190, 176 and backward 535, 523; 4096, backward, 173, 154; 8192
// of 14/2 backward 460, 470; 128 wide, 8192 of 64/8 990, 1150 and backward 3314, 3454; 32 wide
// equal.
template <int D>
constexpr int kRowWaves = D == 64 ? 2 : 1;

template <int D>
int run_fwd(const AttnArgs& in, hipStream_t stream) {
    AttnArgs a = in;
    const bool few = few_rows(a.T, a.hq, D);
    a.tiles = int(tiles_of(a.T, a.cu, a.n_seqs, few ? 64 : 128));
    const int64_t wgs = attn_grid(a.hkv, int64_t(a.tiles) * (a.hq / a.hkv));
    if (int st = check_grid("nf4_attn_fwd", wgs, 256 * kRowWaves<D>); st != NF4_OK) return st;
    if (few)
        hipLaunchKernelGGL((k_attn_fwd<D, 2, 2>), dim3(unsigned(wgs)), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attn_fwd<D, 4, kRowWaves<D>>), dim3(unsigned(wgs)), dim3(256 * kRowWaves<D>), 0, stream, a);
    return check_launch("nf4_attn_fwd");
}

struct BwdGrids {
    bool few, one;         // dq with dk and dv in one launch, of k_attn_bwd_few or _both
    int q_tiles, kv_tiles;
    int64_t q, kv, join;   // workgroups
};

BwdGrids bwd_grids(int64_t T, int64_t hq, int64_t hkv, int64_t D, const void* cu, int64_t n_seqs, int splits) {
    BwdGrids g{};
    g.few = few_tokens(T, n_seqs, hq, hkv), g.one = g.few || one_launch(T, hq);
    g.q_tiles = int(tiles_of(T, cu, n_seqs, 128));
    g.kv_tiles = g.few ? int(tiles_of(T, cu, n_seqs, 32)) : g.q_tiles;
    g.q = attn_grid(int(hkv), int64_t(g.q_tiles) * (hq / hkv));
    g.kv = attn_grid(int(hkv), int64_t(g.kv_tiles) * splits);
    g.join = splits > 1 ? int64_t(g.kv_tiles) * hkv * (kKeyWaves * D / 16) : 0;
    return g;
}

int check_bwd_grids(const char* fn, const BwdGrids& g, int64_t D) {
    int st = g.one ? check_grid(fn, g.q + g.kv, 512) : check_grid(fn, g.q, D == 64 ? 256 * kRowWaves<64> : 256);
    if (st == NF4_OK && !g.one) st = check_grid(fn, g.kv, 512);
    return st == NF4_OK ? check_grid(fn, g.join, 256) : st;
}

template <int D>
int run_bwd(const AttnArgs& in, const BwdGrids& g, hipStream_t stream) {
    AttnArgs a = in;
    a.q_tiles = g.q_tiles, a.tiles = g.kv_tiles;
    if (g.few) {
        hipLaunchKernelGGL(k_attn_bwd_few<D>, dim3(unsigned(g.q + g.kv)), dim3(512), 0, stream, a, unsigned(g.q));
    } else if (g.one) {
        hipLaunchKernelGGL(k_attn_bwd_stats<D>, dim3(unsigned(cdiv(int64_t(a.T) * a.hq * (D / 8), 256))), dim3(256), 0,
                           stream, a);
        const auto both = fine_ds(a.T) ? k_attn_bwd_both<D, true> : k_attn_bwd_both<D, false>;
        hipLaunchKernelGGL(both, dim3(unsigned(g.q + g.kv)), dim3(512), 0, stream, a, unsigned(g.q));
    } else {
        hipLaunchKernelGGL((k_attn_bwd_dq<D, 4, kRowWaves<D>>), dim3(unsigned(g.q)), dim3(256 * kRowWaves<D>), 0, stream, a);
        hipLaunchKernelGGL(k_attn_bwd_dkv<D>, dim3(unsigned(g.kv)), dim3(512), 0, stream, a);
    }
    if (a.splits > 1)
        hipLaunchKernelGGL(k_attn_bwd_join<D>, dim3(unsigned(g.join)), dim3(256), 0, stream, a);
    return check_launch("nf4_attn_bwd");
}

}  // namespace

}  // namespace nf4

using namespace nf4;

extern "C" {

int nf4_attn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t T, int64_t hq, int64_t hkv,
                 int64_t head_dim, const int32_t* cu_seqlens, int64_t n_seqs, int causal, float scale, uint16_t* o,
                 float* lse, nf4_stream stream) {
    const char* fn = "nf4_attn_fwd";
    int st = check_attn(fn, T, hq, hkv, head_dim, cu_seqlens, n_seqs, causal, scale);
    if (st != NF4_OK) return st;
    if (T == 0) return NF4_OK;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !lse ||
        reinterpret_cast<uintptr_t>(lse) % 4 != 0)
        return fail(NF4_E_ARG, "%s: q, k, v and o must be non-NULL and 16-byte aligned, lse 4-byte aligned", fn);
    const size_t q_bytes = size_t(T) * hq * head_dim * 2, k_bytes = size_t(T) * hkv * head_dim * 2;
    const size_t lse_bytes = size_t(T) * hq * 4, cu_bytes = cu_seqlens ? (size_t(n_seqs) + 1) * 4 : 0;
    const ByteRange r[] = {{o, q_bytes}, {lse, lse_bytes}, {q, q_bytes}, {k, k_bytes}, {v, k_bytes}, {cu_seqlens, cu_bytes}};
    if (st = check_apart(fn, r, 2, 6); st != NF4_OK) return st;
    AttnArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = o, a.lse = lse, a.cu = cu_seqlens;
    a.T = int(T), a.n_seqs = int(n_seqs), a.hq = int(hq), a.hkv = int(hkv), a.causal = causal, a.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return head_dim == 128 ? run_fwd<128>(a, s) : head_dim == 64 ? run_fwd<64>(a, s) : run_fwd<32>(a, s);
}

size_t nf4_attn_bwd_workspace(int64_t T, int64_t hq, int64_t hkv, int64_t head_dim, int64_t n_seqs) {
    if (T <= 0 || T > (int64_t(1) << 23) || hkv <= 0 || hq <= 0 || hq % hkv != 0 || hq > 1024 || n_seqs < 0 ||
        n_seqs > kMaxSeqs || (head_dim != 32 && head_dim != 64 && head_dim != 128))
        return 0;
    const AttnBwdPlan p = plan_bwd_attn(T, hq, hkv, head_dim, n_seqs, 1);  // enough with and without a mask
    return p.stats_bytes + std::max(p.part_bytes, plan_bwd_attn(T, hq, hkv, head_dim, n_seqs, 0).part_bytes);
}

int nf4_attn_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const uint16_t* o, const float* lse,
                 const uint16_t* dO, int64_t T, int64_t hq, int64_t hkv, int64_t head_dim, const int32_t* cu_seqlens,
                 int64_t n_seqs, int causal, float scale, uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws,
                 size_t ws_bytes, nf4_stream stream) {
    const char* fn = "nf4_attn_bwd";
    int st = check_attn(fn, T, hq, hkv, head_dim, cu_seqlens, n_seqs, causal, scale);
    if (st != NF4_OK) return st;
    if (T == 0) return NF4_OK;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(dq) ||
        !aligned16(dk) || !aligned16(dv) || !lse || reinterpret_cast<uintptr_t>(lse) % 4 != 0)
        return fail(NF4_E_ARG, "%s: tensors must be non-NULL and 16-byte aligned, lse 4-byte aligned", fn);
    const AttnBwdPlan p = plan_bwd_attn(T, hq, hkv, head_dim, n_seqs, causal);
    const BwdGrids grids = bwd_grids(T, hq, hkv, head_dim, cu_seqlens, n_seqs, p.splits);
    if (st = check_bwd_grids(fn, grids, head_dim); st != NF4_OK) return st;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < p.stats_bytes + p.part_bytes)
        return fail(NF4_E_ARG, "%s: workspace must be 256-byte aligned and at least %zu bytes (got %zu)", fn,
                    p.stats_bytes + p.part_bytes, ws_bytes);
    const size_t q_bytes = size_t(T) * hq * head_dim * 2, k_bytes = size_t(T) * hkv * head_dim * 2;
    const size_t lse_bytes = size_t(T) * hq * 4, cu_bytes = cu_seqlens ? (size_t(n_seqs) + 1) * 4 : 0;
    const ByteRange r[] = {{dq, q_bytes}, {dk, k_bytes}, {dv, k_bytes}, {ws, p.stats_bytes + p.part_bytes}, {q, q_bytes},
                           {k, k_bytes}, {v, k_bytes}, {o, q_bytes}, {dO, q_bytes}, {lse, lse_bytes},
                           {cu_seqlens, cu_bytes}};
    if (st = check_apart(fn, r, 4, 11); st != NF4_OK) return st;
    AttnArgs a{};
    a.q = q, a.k = k, a.v = v, a.o = o, a.dO = dO, a.lse_in = lse, a.dq = dq, a.dk = dk, a.dv = dv, a.cu = cu_seqlens;
    a.T = int(T), a.n_seqs = int(n_seqs), a.hq = int(hq), a.hkv = int(hkv), a.causal = causal, a.scale = scale;
    a.splits = p.splits;
    a.stats = static_cast<float*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.stats_bytes);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return head_dim == 128 ? run_bwd<128>(a, grids, s) : head_dim == 64 ? run_bwd<64>(a, grids, s) : run_bwd<32>(a, grids, s);
}

}  // extern "C"
