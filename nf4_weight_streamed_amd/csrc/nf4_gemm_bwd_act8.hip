// Input gradient and dA of the LoRA linear from an 8-bit checkpoint of its input:
//
//   dX = RNbf( s . g . A + dY . W ),   dA = s . g^T . RNbf(x),   g = dY . B  (fp32, from the pre-pass)
//
// with the NF4 or dense base W.
//
// k_act8_adapter adds g's partials and forms dA, a share per 128 tokens, and s.g as bf16 operands of
// the product: s.g A enters dX as one or two more steps of its contraction, [s.g | dY] . [A ; W].
//
// k_gemm_bwd_act8: a workgroup of eight waves forms a tile of BM x 256 of dX, wave (m, k) its BM/2 x 64.
// Contraction steps of 64: dY is copied straight to LDS a step ahead, dense weights too; NF4 codes are
// loaded two steps ahead and dequantised in registers during the step before theirs. The weight
// tile lies in LDS as in memory, [n][k], and the products' operands come out of it by transposing
// reads. The products are W^T . dY^T, so that a lane holds four neighbours of a row of dX. A wide tile,
// because each weight is then dequantised once per 256 tokens and an operand read from LDS feeds more
// products: 128 x 128 tiles take 325-355 us for 2048 x 8192 x 8192 where these take 262 (dense base) and
// 287 (NF4). Of those 230 and 250 are this kernel's, 1195 and 1100 TFLOP/s; its products and barriers alone,
// without copies and operand reads, take 180, and a large library product of bf16 reaches 1370 TFLOP/s. 56 %
// of the cycles have a matrix instruction under way (NF4 in the loop's first form: 42 %).
// 512 x 18944 x 3584 with NF4 (a 7B gate projection's backward) takes 103-105 us in a row; a kernel trace, one launch at a
// time, has 14 for g and dB, 6 for the adapter, 74-76 here, 13 for the sums of the pieces, whose 2 x 66 MB are the price of
// cutting 28 tiles for 256 CUs. 1291 x 5120 x 5120 dense: 100-105.
#include "act8.h"
#include "common.h"
#include "device.h"
#include "shares.h"

namespace nf4 {

namespace {

constexpr int kBN = 64;        // contraction per step
constexpr int kBK = 256;       // dX columns of a tile
constexpr int kThreads = 512;
constexpr int kBT = 128;       // tokens of a share of dA
constexpr int kCols = 128;     // its columns at a time
constexpr int64_t kCUs = kChipCUs;

// What the plan weighs, in steps of a 256 x 256 tile (1.8 us with a dense base, 2.0 with NF4, all CUs at work):
// a step of a 128 x 256 tile, a tile's sums written and read again (14 steps for 256 of them), and the launch that
// reads them, where dA has one share and it reads nothing else. The narrower tile costs more where its weights take
// decoding or come from memory: a dense base of 283 MB, 245 tokens, 134 us in tiles of 128 tokens, 115 in 256;
// one of 52 MB, 1291 tokens, 105 and 107. Over 88 sizes (40 to 3000 tokens, both bases) the choice is
// within 6 % of the best of both tiles and all cuts.
constexpr double kStep128 = 0.57, kStep128Far = 0.75, kSlot = 14.0 / kCUs, kLaunch = 2.0;
constexpr int64_t kLastLevelCache = int64_t(256) << 20;

// The adapter's steps: s.g as hi and lo parts of 32 ranks each side by side, or of 64 each in steps of their own.
__host__ __device__ constexpr int adapter_steps(int r) { return r == 0 ? 0 : r <= 32 ? 1 : 2; }

// Whole tiles, a multiple of the CUs, and a tail whose contraction is cut into pieces of `per` steps (in
// one: whole tiles too). Workgroup w takes piece w / tail of tile w % tail, so that the workgroups of an
// XCD read the same rows of W and columns of dY at about the same time; their sums lie in slot w. (Equal
// runs of steps from tile to tile balance better, but their neighbours share nothing: 512 x 18944 x
// 3584 119 against 109 us, 1291 x 5120 x 5120 with a dense base 128 against 106.)
struct WideTiles {
    int full, tail, pieces, per;  // pieces: of the tail together
    int steps, mtiles;            // contraction steps; token tiles (tile = token tile + mtiles * column tile)
};

// s.g and dA's shares. Block c + chunks m: columns [c, c + 1) 128 cols of K, tokens [m, m + 1) 128. Latency
// bounds it: loads are issued early, and eight waves share a block's instructions. kRanks: r at most.
template <int kRanks>
__global__ __launch_bounds__(kThreads, 2) void k_act8_adapter(const float* __restrict__ gpart, int parts,
                                                              const uint8_t* __restrict__ x, const float* __restrict__ x_scale,
                                                              int T, int K, int r, float s, int cols, int chunks,
                                                              uint16_t* __restrict__ sg, float* __restrict__ dapart) {
    constexpr int kTP = kBT + 8;  // pitch of the [.][t] tiles
    __shared__ __align__(16) uint16_t sg_hi[kRanks * kTP], sg_lo[kRanks * kTP], sg_rest[kRanks * kTP], sxt[kCols * kTP];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int chunk = int(blockIdx.x) % chunks, tm = int(blockIdx.x) / chunks;
    const int m0 = tm * kBT, k0 = chunk * cols * kCols, k1 = min(K, k0 + cols * kCols);
    const uint32_t trows = uint32_t(min(kBT, T - m0));
    const int rp = (r + 15) & ~15, half = r <= 32 ? 32 : 64;
    const auto rx = make_rsrc(x + size_t(m0) * K, trows * uint32_t(K));
    const auto rxs = make_rsrc(x_scale + size_t(m0) * (K / 64), trows * uint32_t(K / 64) * 4u);
    // x: thread (column octet, token group) takes 8 columns of kXT tokens; rows past T read as zeros, columns
    // past K are the next row's and their sums are not stored
    constexpr int kXT = kBT / 32;
    const int xk8 = 8 * (tid & 15), xt0 = kXT * (tid >> 4);
    u32x2 xc[kXT];
    float xs[kXT];
    auto load_x = [&](int k) {
#pragma unroll
        for (int i = 0; i < kXT; ++i) {
            const uint32_t at = uint32_t(xt0 + i) * uint32_t(K) + uint32_t(k + xk8);
            xc[i] = buf_load8(rx, at);
            xs[i] = buf_load_f32(rxs, at / 64 * 4u);
        }
    };
    auto stage_x = [&]() {
        u32x4 v[kXT];
#pragma unroll
        for (int i = 0; i < kXT; ++i) {
            float f[8];
            act8_values8(xc[i], xs[i], f);
            v[i] = pack_octet(f);
        }
        // token t of column k lies at t ^ (k & ~7): the octets' stores do not meet in a bank
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // element e of tokens 2 p and 2 p + 1: low halves (e even) or high halves (e odd)
            const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
            u32x2 t;
#pragma unroll
            for (int p = 0; p < kXT / 2; ++p) t[p] = __builtin_amdgcn_perm(v[2 * p + 1][e >> 1], v[2 * p][e >> 1], sel);
            *reinterpret_cast<u32x2*>(&sxt[(xk8 + e) * kTP + (xt0 ^ xk8)]) = t;
        }
    };
    load_x(k0);
    // g, thread (token, 4 ranks) for 16 ranks at a time: its partials in their order, all loads under way at once.
    // One descriptor per partial over this tile's rows; 12 bytes of slack keep the last 16-byte load
    // (4-byte aligned, ranks >= r masked below) inside it, and inside the allocation: the partials
    // region is padded to 256 bytes. s.g as three bf16 parts, planes [rank][t]: dA is off by fp32's
    // roundings alone (with two parts, by 2^-17 of each term); dX, rounded to bf16, takes hi and lo.
    const int gt = tid / 4;
    const uint32_t gbytes = trows * uint32_t(r) * 4u + 12u;
    const size_t gstride = size_t(T) * r;
    for (int j0 = 0; j0 < half; j0 += 16) {
        const int j = j0 + 4 * (tid % 4);
        u32x2 h = {0, 0}, l = {0, 0};
        if (j0 < r) {
            const uint32_t at = m0 + gt < T && j < r ? (uint32_t(gt) * uint32_t(r) + uint32_t(j)) * 4u : kOutOfRange;
            f32x4 pv[kMaxGParts];
            const float* from = gpart + size_t(m0) * r;
#pragma unroll
            for (int p = 0; p < kMaxGParts; ++p) {
                pv[p] = __builtin_bit_cast(f32x4, buf_load16(make_rsrc(from, gbytes), p < parts ? at : kOutOfRange));
                if (p + 1 < parts) from += gstride;
            }
            f32x4 g = pv[0];
#pragma unroll
            for (int p = 1; p < kMaxGParts; ++p)
                if (p < parts) g += pv[p];
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                __bf16 hh, ll, rr;
                split_bf16(j + c < r ? s * g[c] : 0.0f, hh, ll, rr);
                hi[c] = __builtin_bit_cast(uint16_t, hh), lo[c] = __builtin_bit_cast(uint16_t, ll);
                sg_hi[(j + c) * kTP + gt] = hi[c];
                sg_lo[(j + c) * kTP + gt] = lo[c];
                sg_rest[(j + c) * kTP + gt] = __builtin_bit_cast(uint16_t, rr);
            }
            h = u32x2{hi[0] | uint32_t(hi[1]) << 16, hi[2] | uint32_t(hi[3]) << 16};
            l = u32x2{lo[0] | uint32_t(lo[1]) << 16, lo[2] | uint32_t(lo[3]) << 16};
        }
        if (chunk == 0 && sg && m0 + gt < T) {
            uint16_t* to = sg + size_t(m0 + gt) * 2 * half + j;
            *reinterpret_cast<u32x2*>(to) = h;
            *reinterpret_cast<u32x2*>(to + half) = l;
        }
    }

    // D[k][j] over t, 16x16x32 MFMAs: a wave owns 16 of the 128 staged columns
    const int l16 = lane & 15, t8 = 8 * (lane >> 4);
    float* dpart = dapart + size_t(tm) * r * K;
    for (int k = k0; k < k1; k += kCols) {
        if (k > k0) __syncthreads();  // the columns before have been read
        stage_x();
        if (k + kCols < k1) load_x(k + kCols);
        __syncthreads();
        for (int jb = 0; jb < rp / 16; ++jb) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ts = 0; ts < kBT / 32; ++ts) {
                const int tt = 32 * ts + t8, c = 16 * wave + l16;
                const bf16x8 xa = as_bf16x8(*reinterpret_cast<const u32x4*>(&sxt[c * kTP + (tt ^ (c & ~7))]));
                const int g = (16 * jb + l16) * kTP + tt;
                d = mfma16x16x32(xa, as_bf16x8(*reinterpret_cast<const u32x4*>(&sg_hi[g])), d);
                d = mfma16x16x32(xa, as_bf16x8(*reinterpret_cast<const u32x4*>(&sg_lo[g])), d);
                d = mfma16x16x32(xa, as_bf16x8(*reinterpret_cast<const u32x4*>(&sg_rest[g])), d);
            }
            // lane holds D[column 16 wave + 4 (lane / 16) + e][j = 16 jb + lane % 16]
            const int j = 16 * jb + l16, kq = k + 16 * wave + 4 * (lane >> 4);
            if (j < r && kq < k1) *reinterpret_cast<f32x4*>(&dpart[size_t(j) * K + kq]) = d;
        }
    }
}

template <int BM, bool kDense>
__global__ __launch_bounds__(kThreads, 2) void k_gemm_bwd_act8(const uint16_t* __restrict__ dy, const void* __restrict__ weights,
                                                               const float* __restrict__ absmax, const uint16_t* __restrict__ sg,
                                                               const uint16_t* __restrict__ A, int T, int N, int K, int r,
                                                               WideTiles tl, uint16_t* __restrict__ dx, float* __restrict__ partial,
                                                               Tables tab) {
    constexpr int WM = BM / 2, FM = WM / 32, FK = 2;
    // two dY and two weight tiles, each a variable of its own: the compiler then knows that reads of one
    // do not wait for copies into another
    __shared__ __align__(1024) uint16_t sA0[BM * kBN], sW0[kBN * kBK], sA1[BM * kBN], sW1[kBN * kBK];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wk = wave & 3;
    const int frag_row = lane & 31;
    // the weights of the whole matrix (the entry points keep their bytes below 2^31); rows beyond N load as
    // zeros. Columns beyond K of a ragged tile read the next row's data: they only reach dX columns
    // that are never stored.
    const auto rcd = make_rsrc(weights, uint32_t(N) * uint32_t(K) * (kDense ? 2u : 1u) / (kDense ? 1u : 2u));
    const int ext = adapter_steps(r);
    const auto ra = make_rsrc(A, uint32_t(r) * uint32_t(K) * 2u);  // rows at or beyond r read as zeros
    const auto rsc = make_rsrc(kDense ? nullptr : absmax, kDense ? 0u : uint32_t(N) * uint32_t(K / 64) * 4u);

    // dY tile [BM][64]: 128-byte rows, the 16-byte chunk c of row r at c ^ ((r / 2) % 8). A copy instruction of a
    // wave fills 8 rows, its lanes picking the global chunk that belongs where they write.
    constexpr int kPiecesA = BM / 64;
    const int a_row = lane >> 3, a_chunk = (lane & 7) ^ (lane >> 4);
    auto stage_rows = [&](const __amdgpu_buffer_rsrc_t& from, int nb, uint32_t stride, uint16_t* to) {
#pragma unroll
        for (int i = 0; i < kPiecesA; ++i) {
            const int p = kPiecesA * wave + i;
            // columns at or beyond the stride (ragged last step) load as zeros
            const uint32_t n = uint32_t(nb * kBN) + 8u * uint32_t(a_chunk ^ ((p & 1) << 2));
            const uint32_t off = (uint32_t(8 * p + a_row) * stride + n) * 2u;
            buf_load16_lds(from, n < stride ? off : kOutOfRange, to + 512 * p);
        }
    };
    // Weight tile [64][256]: 512-byte rows in two lines of 16 chunks; a chunk's place in its line is its number
    // ^ swizzle(n) ^ 2 in the second line. A transposing read takes one 64-byte segment of four rows and a
    // store of dequantised chunks eight rows' every fourth chunk: no conflicts are counted for the reads, eight
    // cycles for a store (of 16).
    auto swizzle = [](int n) { return ((n & 3) << 2) | ((n ^ (n >> 2)) & 3); };
    auto stage_w = [&](const __amdgpu_buffer_rsrc_t& from, int k0, int n0, int row_mask, uint16_t* to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = 4 * wave + i, row = 2 * p + (lane >> 5), place = lane & 31;
            const int c = place ^ swizzle(row) ^ ((place >> 4) << 1);
            buf_load16_lds(from, (uint32_t(n0 + (row & row_mask)) * uint32_t(K) + uint32_t(k0 + 8 * c)) * 2u, to + 512 * p);
        }
    };
    // NF4: thread (row, eighth) loads 32 codes and their scale ...
    struct Codes {
        u32x4 c;
        float s;
    };
    const int w_row = tid >> 3, w_q = tid & 7;
    auto load_codes = [&](int k0, int nb, Codes& l) {
        const uint32_t n = uint32_t(nb * kBN + w_row), k = uint32_t(k0 + 32 * w_q);
        l.c = buf_load16(rcd, n * uint32_t(K / 2) + k / 2);
        l.s = buf_load_f32(rsc, (n * uint32_t(K / 64) + k / 64) * 4u);
    };
    // ... and stores them as bf16: the 16 scaled levels once, as two tables of bytes in registers, then a
    // byte permute of each table's halves for four codes at a time: no reads of LDS, which the products'
    // operands keep busy
    uint32_t lo[4], hi[4];
    auto scale_levels = [&](float scale) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // level * absmax in fp32, then RNbf: the format's two roundings
            const uint32_t p = pack_bf16x2(tab.level[4 * i] * scale, tab.level[4 * i + 1] * scale);
            const uint32_t q = pack_bf16x2(tab.level[4 * i + 2] * scale, tab.level[4 * i + 3] * scale);
            lo[i] = __builtin_amdgcn_perm(q, p, 0x06040200u);
            hi[i] = __builtin_amdgcn_perm(q, p, 0x07050301u);
        }
    };
    const int w_swizzle = swizzle(w_row) ^ ((w_q >> 2) << 1);
    auto store_codes = [&](uint32_t c, int e, uint16_t* to) {  // 8 codes: even ones in the low nibbles
        auto four = [&](uint32_t s) {  // bytes of s: codes 0..15
            const uint32_t at = s & 0x07070707u;
            // permute selectors 12 and 13 give the bytes 0 and 255: the upper half's mask
            const uint32_t up = __builtin_amdgcn_perm(0u, 0u, ((s >> 3) & 0x01010101u) | 0x0C0C0C0Cu);
            const uint32_t l0 = __builtin_amdgcn_perm(lo[1], lo[0], at), l1 = __builtin_amdgcn_perm(lo[3], lo[2], at);
            const uint32_t h0 = __builtin_amdgcn_perm(hi[1], hi[0], at), h1 = __builtin_amdgcn_perm(hi[3], hi[2], at);
            const uint32_t lb = (l1 & up) | (l0 & ~up), hb = (h1 & up) | (h0 & ~up);
            return u32x2{__builtin_amdgcn_perm(hb, lb, 0x05010400u), __builtin_amdgcn_perm(hb, lb, 0x07030602u)};
        };
        const uint32_t even = c & 0x0F0F0F0Fu, odd = (c >> 4) & 0x0F0F0F0Fu;
        const u32x2 x = four(__builtin_amdgcn_perm(odd, even, 0x05010400u));
        const u32x2 y = four(__builtin_amdgcn_perm(odd, even, 0x07030602u));
        *reinterpret_cast<u32x4*>(to + w_row * kBK + (((4 * w_q + e) ^ w_swizzle) << 3)) = u32x4{x.x, x.y, y.x, y.y};
    };

    // Fragment addresses (bytes). dY: row wm WM + 32 i + lane % 32, chunk 2 kk + lane / 32. Weights: two
    // transposing reads of four rows each, rows 16 kk + 8 (lane / 32) + 4 t + (lane % 16) / 4, columns
    // 64 wk + 32 j + 16 ((lane / 16) % 2) + lane % 16. swizzle(n) of those rows: n / 4 % 4 = 2 (lane / 32) + t.
    uint32_t w_at[FK][2];
    const uint32_t a_at = uint32_t((wm * WM + frag_row) * 128 + (((lane >> 5) ^ ((frag_row >> 1) & 7)) << 4));  // kk = 0; ^ 32 kk
#pragma unroll
    for (int j = 0; j < FK; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int n = 8 * (lane >> 5) + 4 * t + ((lane & 15) >> 2);
            const int c = 8 * wk + 4 * j + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            w_at[j][t] = uint32_t(n * 2 * kBK + ((c ^ swizzle(n) ^ ((wk >> 1) << 1)) << 4) + (lane & 1) * 8);
        }

    f32x16 acc[FM][FK];
    bf16x8 af[2][FM], bw[2][FK];  // operands of one 16-deep product and the next
    auto read_frags = [&](const uint16_t* a_tile, const uint16_t* w_tile, int set, int kk) {
        const char *at = reinterpret_cast<const char*>(a_tile), *wt = reinterpret_cast<const char*>(w_tile);
#pragma unroll
        for (int j = 0; j < FK; ++j)
            bw[set][j] = lds_frag_tr(wt + w_at[j][0] + 32 * kBK * kk, wt + w_at[j][1] + 32 * kBK * kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
            af[set][i] = as_bf16x8(*reinterpret_cast<const u32x4*>(at + (a_at ^ uint32_t(kk << 5)) + 32 * 128 * i));
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FK; ++j) acc[i][j] = mfma32x32x16(bw[set][j], af[set][i], acc[i][j]);
    };

    // Whole tiles, a round of the CUs after the other, then the pieces: steps [s0, s1) of a tile
    const int b = int(blockIdx.x);
    int tile, s0 = 0, s1 = tl.steps, w = 0;
    if (b < tl.full) {
        tile = b / int(kCUs) * int(kCUs) + int(xcd_tile_order(uint32_t(b) % uint32_t(kCUs), uint32_t(kCUs)));
    } else {
        w = int(xcd_tile_order(uint32_t(b - tl.full), uint32_t(tl.pieces)));
        tile = tl.full + w % tl.tail;
        s0 = w / tl.tail * tl.per;
        s1 = min(tl.steps, s0 + tl.per);
    }
    const int tm = tile % tl.mtiles, k0 = tile / tl.mtiles * kBK, m0 = tm * BM;
    const uint32_t trows = uint32_t(min(BM, T - m0));
    const auto rdy = make_rsrc(dy + size_t(m0) * N, trows * uint32_t(N) * 2u);
    auto stage = [&](int nb, uint16_t* a, uint16_t* wt) {  // what is copied of step nb's tiles
        stage_rows(rdy, nb, uint32_t(N), a);
        if constexpr (kDense) stage_w(rcd, k0, nb * kBN, 63, wt);
    };
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    Codes ld[2];
    stage(s0, sA0, sW0);
    if constexpr (!kDense) {
        load_codes(k0, s0, ld[0]);
        load_codes(k0, s0 + 1, ld[1]);
    }
    if (s0 == 0) {  // s.g A
        const auto rsg = make_rsrc(sg + size_t(m0) * (64 * ext), trows * uint32_t(64 * ext) * 2u);
        for (int x = 0; x < ext; ++x) {
            stage_rows(rsg, x, uint32_t(64 * ext), sA1);
            stage_w(ra, k0, 0, ext == 1 ? 31 : 63, sW1);
            wait_vmcnt<0>();
            __syncthreads();
            for (int kk = 0; kk < kBN / 16; kk += 2) {
                read_frags(sA1, sW1, 0, kk);
                read_frags(sA1, sW1, 1, kk + 1);
                multiply(0);
                multiply(1);
            }
            __syncthreads();  // the next copies take their place
        }
    }
    // Step nb's last products run after the barrier that tells that every wave has read its tiles and that
    // the next step's are there: copies into their place start then, a step ahead of their use, and the
    // next step's first operands are read beside them. Codes are dequantised between the products.
    if (s0 + 1 < s1) stage(s0 + 1, sA1, sW1);
    if constexpr (!kDense) {
        scale_levels(ld[0].s);
#pragma unroll
        for (int e = 0; e < 4; ++e) store_codes(ld[0].c[e], e, sW0);
        load_codes(k0, s0 + 2, ld[0]);
        scale_levels(ld[1].s);
    }
    wait_vmcnt<0>();
    __syncthreads();
    read_frags(sA0, sW0, 0, 0);
    auto step = [&](int nb, Codes& now, Codes& then, uint16_t* a, uint16_t* wt, const uint16_t* a_next, uint16_t* w_next) {
        read_frags(a, wt, 1, 1);
        if constexpr (!kDense) store_codes(now.c[0], 0, w_next);
        multiply(0);
        read_frags(a, wt, 0, 2);
        if constexpr (!kDense) store_codes(now.c[1], 1, w_next), store_codes(now.c[2], 2, w_next);
        multiply(1);
        read_frags(a, wt, 1, 3);
        if constexpr (!kDense) store_codes(now.c[3], 3, w_next);
        multiply(0);
        wait_vmcnt<0>();
        __syncthreads();
        if (nb + 2 < s1) stage(nb + 2, a, wt);
        if constexpr (!kDense) load_codes(k0, nb + 3, now);  // past the end: zeros, or codes that nothing uses
        read_frags(a_next, w_next, 0, 0);
        if constexpr (!kDense) scale_levels(then.s);
        multiply(1);
    };
    for (int nb = s0;;) {
        step(nb, ld[1], ld[0], sA0, sW0, sA1, sW1);
        if (++nb == s1) break;
        step(nb, ld[0], ld[1], sA1, sW1, sA0, sW0);
        if (++nb == s1) break;
    }

    // acc[i][j][4 q + e] is token wm WM + 32 i + lane % 32, column 64 wk + 32 j + 8 q + 4 (lane / 32) + e
    if (s0 == 0 && s1 == tl.steps) {
        if (k0 + 64 * wk < K) {  // K % 64 == 0
            const auto rdx = make_rsrc(dx + size_t(m0) * K, trows * uint32_t(K) * 2u);  // rows past T are dropped
            const uint32_t at = (uint32_t(wm * WM + frag_row) * uint32_t(K) + uint32_t(k0 + 64 * wk) + 4u * (lane >> 5)) * 2u;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FK; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        __builtin_amdgcn_raw_buffer_store_b64(
                            u32x2{pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                                  pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])},
                            rdx, int(at + uint32_t(32 * i) * uint32_t(K) * 2u + uint32_t(32 * j + 8 * q) * 2u), 0, 0);
        }
    } else {
        float* to = partial + size_t(w) * (BM * kBK) + wave * (FM * FK * 1024) + lane * 4;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FK; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4*>(to + (i * FK + j) * 1024 + q * 256) =
                        f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
}

// dX = RNbf(sum of the pieces' sums) of the tail's cut tiles, four elements a thread; then the sums of dA's and
// dB's shares.
template <int BM>
__global__ __launch_bounds__(256) void k_gemm_bwd_act8_finish(const float* __restrict__ partial, WideTiles tl, int T, int K,
                                                              uint16_t* __restrict__ dx, int64_t dx_blocks, Shares da,
                                                              int64_t da_blocks, Shares db) {
    const int64_t b = blockIdx.x;
    if (b >= dx_blocks) {
        b < dx_blocks + da_blocks ? sum_shares(da, b - dx_blocks) : sum_shares(db, b - dx_blocks - da_blocks);
        return;
    }
    constexpr int kBlocks = BM * kBK / 1024;  // of a tile
    const int q = int(b / kBlocks), loc = (int(b % kBlocks) * 256 + int(threadIdx.x)) * 4;
    // the place of these four in the tile: see the end of k_gemm_bwd_act8
    constexpr int FM = BM / 64;
    const int lane = loc / 4 % 64, sub = loc / 256 % 4, j = loc / 1024 % 2, i = loc / 2048 % FM, wave = loc / (2048 * FM);
    const int tile = tl.full + q, row = tile % tl.mtiles * BM + (wave >> 2) * (BM / 2) + 32 * i + lane % 32;
    const int col = tile / tl.mtiles * kBK + 64 * (wave & 3) + 32 * j + 8 * sub + 4 * (lane >> 5);
    if (row >= T || col >= K) return;  // K % 64 == 0: the four columns are all in or all out
    const f32x4 a = sum_slots(partial + size_t(q) * (BM * kBK) + loc, tl.pieces / tl.tail, size_t(tl.tail) * (BM * kBK));
    *reinterpret_cast<u32x2*>(dx + size_t(row) * K + col) = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
}

}  // namespace

BwdPlan plan_bwd_act8(int64_t T, int64_t N, int64_t K, int r, bool dense) {
    if (T <= kSkinnyBwdT && !dense) return plan_bwd(T, N, K, r, dense);
    BwdPlan p{};
    double best = 0;
    const int64_t steps = cdiv(N, kBN);
    for (int bm : {128, 256}) {
        const double step = bm == 256 ? 1.0 : dense && N * K * 2 <= kLastLevelCache ? kStep128 : kStep128Far, slot = kSlot * bm / 256;
        const int64_t tiles = cdiv(T, bm) * cdiv(K, kBK), full = tiles / kCUs * kCUs, tail = tiles - full;
        for (int64_t cut = 1; cut <= (tail > 0 ? std::min(kCUs / tail, steps) : 1); ++cut) {
            const int64_t per = tail > 0 ? cdiv(steps, cut) : 0, pieces = tail > 0 ? cdiv(steps, per) * tail : 0;
            const double cost = double(full / kCUs * steps + per) * step + (pieces > tail ? slot * double(pieces) + (T <= kBT ? kLaunch : 0.0) : 0.0);
            if (best > 0 && cost >= best) continue;
            best = cost;
            p.bm = bm;
            p.bn = kBK;
            p.mtiles = int(cdiv(T, bm));
            p.ktiles = int(cdiv(K, kBK));
            p.full = int(full);
            p.tail = int(tail);
            p.pieces = int(pieces);
            p.steps_per_piece = int(per);
        }
    }
    if (r > 0) plan_lora_bwd_pre(p, T, N, kMaxGParts);
    size_t off = 0;
    p.off_gpart = off;
    off += align256(size_t(p.gparts) * size_t(T) * size_t(r) * 4);
    p.off_dapart = off;
    off += r > 0 && T > kBT ? align256(size_t(cdiv(T, kBT)) * size_t(r) * size_t(K) * 4) : 0;
    p.off_dbpart = off;
    off += r > 0 && p.dbchunks > 1 ? align256(size_t(p.dbchunks) * size_t(N) * size_t(r) * 4) : 0;
    p.off_sg = off;
    off += align256(size_t(T) * size_t(64 * adapter_steps(r)) * 2);
    p.off_dx = off;
    off += p.pieces > p.tail ? size_t(p.pieces) * size_t(p.bm) * size_t(p.bn) * 4 : 0;
    p.ws_bytes = std::max<size_t>(off, 256);  // never none
    return p;
}

hipError_t launch_gemm_bwd_act8(const BwdPlan& p, const uint8_t* codes, const float* absmax, const uint16_t* wdense,
                                const uint16_t* dy, const SavedInput& x, const uint16_t* A, int64_t T, int64_t N,
                                int64_t K, int r, float s, uint16_t* dx, float* dA, float* dB, void* ws,
                                hipStream_t stream) {
    char* w = static_cast<char*>(ws);
    const WideTiles tl{p.full, p.tail, p.pieces, p.steps_per_piece, int(cdiv(N, kBN)), p.mtiles};
    float* partial = dx && tl.pieces > tl.tail ? reinterpret_cast<float*>(w + p.off_dx) : nullptr;
    float* dapart = cdiv(T, kBT) == 1 ? dA : reinterpret_cast<float*>(w + p.off_dapart);
    uint16_t* sg = reinterpret_cast<uint16_t*>(w + p.off_sg);
    const int shares = int(cdiv(T, kBT));
    if (r > 0) {
        // about one workgroup a CU: each adds g's partials of its tokens for itself
        const int64_t groups = cdiv(K, kCols), cols = std::max<int64_t>(1, cdiv(shares * groups, kCUs));
        const int64_t chunks = cdiv(groups, cols);
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(unsigned(chunks * shares)), dim3(kThreads), 0, stream,
                               reinterpret_cast<const float*>(w + p.off_gpart), p.gparts, x.codes, x.scale, int(T), int(K), r, s,
                               int(cols), int(chunks), dx ? sg : nullptr, dapart);
        };
        launch(r <= 16 ? k_act8_adapter<16> : k_act8_adapter<64>);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dx) {
        prof_gemm_begin(stream);
        auto launch = [&](auto kernel, const void* weights) {
            hipLaunchKernelGGL(kernel, dim3(unsigned(tl.full + tl.pieces)), dim3(kThreads), 0, stream, dy, weights, absmax,
                               sg, A, int(T), int(N), int(K), r, tl, dx, partial, tables());
        };
        if (wdense)
            launch(p.bm == 256 ? k_gemm_bwd_act8<256, true> : k_gemm_bwd_act8<128, true>, wdense);
        else
            launch(p.bm == 256 ? k_gemm_bwd_act8<256, false> : k_gemm_bwd_act8<128, false>, codes);
        prof_gemm_end(stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const Shares da{dapart, shares, r > 0 && shares > 1 ? int64_t(r) * K : 0, dA};
    // dB shares (N * r is a multiple of 4: N % 16 == 0)
    const Shares db{reinterpret_cast<const float*>(w + p.off_dbpart), p.dbchunks, r > 0 && p.dbchunks > 1 ? N * r : 0, dB};
    const int64_t dx_blocks = partial ? int64_t(p.tail) * (p.bm * p.bn / 1024) : 0;
    const int64_t da_blocks = cdiv(da.total / 4, 256), db_blocks = cdiv(db.total / 4, 256);
    if (dx_blocks + da_blocks + db_blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((p.bm == 256 ? k_gemm_bwd_act8_finish<256> : k_gemm_bwd_act8_finish<128>),
                       dim3(unsigned(dx_blocks + da_blocks + db_blocks)), dim3(256), 0, stream, partial, tl, int(T), int(K), dx,
                       dx_blocks, da, da_blocks, db);
    return hipGetLastError();
}

}  // namespace nf4
