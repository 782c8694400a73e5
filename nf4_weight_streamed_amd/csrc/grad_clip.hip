// Global gradient norm over many tensors, and clipping: with all the elements g of a list,
//   n = sqrt(sum g^2),   out = g * min(1, max_norm / (n + 10^-6)).
// Memory bound: g is read for the norm, then read and written for the scaling (not at all
// where it is in place and nothing has to be scaled). The scaling goes from the last element
// to the first, so that it finds in the last-level cache what the norm read last; in lists
// larger than that cache the rest is read and the outputs are written past it: 842 MB of fp32
// (1120 tensors) 497 -> 422 us, 6.0 TB/s of the three passes' bytes (norm 123 us, 6.8 TB/s); in
// place 428 us; of bf16 (421 MB) 210 us.
// Squares and their sums are fp64, at the full rate of the vector ALUs beside these loads: no
// overflow or underflow for any fp32 gradient, and sums over 10^9 elements stay exact far below
// the fp32 result's rounding. No atomics: every workgroup leaves one fp64 share, and every
// workgroup of the scaling launch sums the shares itself, in the same order, instead of a third
// launch.
#include <algorithm>
#include <cmath>
#include <iterator>
#include <new>
#include <utility>
#include <vector>

#include "../../include/nf4lora.h"
#include "common.h"
#include "device.h"

namespace nf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxShares = 1024;
constexpr double kCacheBytes = 192e6;  // of the 256 MB last-level cache, what a pass leaves to the next

// One piece of one tensor; pieces of a list cover its elements once. kWide pieces start
// 16-byte aligned in both buffers.
struct Chunk {
    const void* in;
    void* out;
    uint32_t count;
    uint32_t flags;
    uint64_t pad;
};
constexpr uint32_t kBf16 = 1, kWide = 2;
static_assert(sizeof(Chunk) == 32, "two 16-byte reads");

__device__ __forceinline__ double block_sum(double v, double* red) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((red[0] + red[1]) + red[2]) + red[3];
}

__device__ __forceinline__ double sq(float v) { return double(v) * double(v); }

__device__ __forceinline__ double sq16(u32x4 v, bool bf16) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (bf16)
            s += sq(__uint_as_float(v[e] << 16)) + sq(__uint_as_float(v[e] & 0xFFFF0000u));
        else
            s += sq(__uint_as_float(v[e]));
    }
    return s;
}

// Non-temporal for what the caches would not keep until it is wanted again; at compile time,
// a choice at run time beside each access cost the gain.
template <bool NT>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
    return NT ? __builtin_nontemporal_load(p) : *p;
}

template <bool NT>
__device__ __forceinline__ double chunk_sum(const Chunk ch) {
    const bool bf16 = ch.flags & kBf16;
    const uint32_t per = bf16 ? 8 : 4;
    const uint32_t wide = (ch.flags & kWide) ? ch.count / per : 0;
    const u32x4* p = static_cast<const u32x4*>(ch.in);
    double sum = 0.0;
    uint32_t i = threadIdx.x;
    for (; i + 3 * kThreads < wide; i += 4 * kThreads) {
        u32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = load16<NT>(p + i + u * kThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u) sum += sq16(v[u], bf16);
    }
    for (; i < wide; i += kThreads) sum += sq16(p[i], bf16);
    for (uint32_t e = wide * per + threadIdx.x; e < ch.count; e += kThreads)
        sum += sq(bf16 ? bf16_to_f32(static_cast<const uint16_t*>(ch.in)[e]) : static_cast<const float*>(ch.in)[e]);
    return sum;
}

// Pieces below `stream` are read past the caches, so that these hold the others when the
// scaling launch starts there.
__global__ __launch_bounds__(kThreads) void k_grad_norm(const Chunk* __restrict__ chunks, int n, int stream,
                                                        double* __restrict__ shares) {
    __shared__ double red[4];
    double sum = 0.0;
    for (int c = blockIdx.x; c < n; c += gridDim.x)
        sum += c < stream ? chunk_sum<true>(chunks[c]) : chunk_sum<false>(chunks[c]);
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) shares[blockIdx.x] = sum;
}

// The factor stays fp64: as fp32 it would lose bits below 2^-126, which bounds far below the norm reach.
// bf16 is rounded by way of fp32.
__device__ __forceinline__ float scaled(float v, double f) { return float(double(v) * f); }

__device__ __forceinline__ u32x4 scale16(u32x4 v, double f, bool bf16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (bf16)
            v[e] = pack_bf16x2(scaled(__uint_as_float(v[e] << 16), f), scaled(__uint_as_float(v[e] & 0xFFFF0000u), f));
        else
            v[e] = __float_as_uint(scaled(__uint_as_float(v[e]), f));
    }
    return v;
}

template <bool LOAD_NT, bool STORE_NT>
__device__ __forceinline__ void chunk_scale(const Chunk ch, double f) {
    const bool bf16 = ch.flags & kBf16;
    const uint32_t per = bf16 ? 8 : 4;
    const uint32_t wide = (ch.flags & kWide) ? ch.count / per : 0;
    const u32x4* p = static_cast<const u32x4*>(ch.in);
    u32x4* d = static_cast<u32x4*>(ch.out);
    uint32_t i = threadIdx.x;
    for (; i + 3 * kThreads < wide; i += 4 * kThreads) {
        u32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = load16<LOAD_NT>(p + i + u * kThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const u32x4 w = scale16(v[u], f, bf16);
            if constexpr (STORE_NT)
                __builtin_nontemporal_store(w, d + i + u * kThreads);
            else
                d[i + u * kThreads] = w;
        }
    }
    for (; i < wide; i += kThreads) d[i] = scale16(p[i], f, bf16);
    for (uint32_t e = wide * per + threadIdx.x; e < ch.count; e += kThreads) {
        if (bf16)
            static_cast<uint16_t*>(ch.out)[e] = bf16_bits(scaled(bf16_to_f32(static_cast<const uint16_t*>(ch.in)[e]), f));
        else
            static_cast<float*>(ch.out)[e] = scaled(static_cast<const float*>(ch.in)[e], f);
    }
}

// The norm from the shares (written by workgroup 0); then, when `scale`, the pieces, from the
// last one on. A norm that is not finite scales by 1: the caller sees it in *norm.
__global__ __launch_bounds__(kThreads) void k_grad_scale(const Chunk* __restrict__ chunks, int n,
                                                         const double* __restrict__ shares, int n_shares,
                                                         float max_norm, int scale, int in_place, int stream,
                                                         float* __restrict__ norm) {
    __shared__ double red[4];
    double sum = 0.0;
    for (int i = threadIdx.x; i < n_shares; i += kThreads) sum += shares[i];
    const double total = sqrt(block_sum(sum, red));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = float(total);
    if (!scale) return;
    const double q = double(max_norm) / (total + 1e-6);
    const bool clip = q < 1.0 && total < __builtin_inf();
    if (in_place && !clip) return;
    const double f = clip ? q : 1.0;
    int c = n - 1 - int(blockIdx.x);
    auto leave = [&](const Chunk& ch) { return !clip && ch.in == ch.out; };  // in place, among others that are not
    for (; c >= stream; c -= gridDim.x) {
        const Chunk ch = chunks[c];
        if (leave(ch)) continue;
        if (stream == 0)
            chunk_scale<false, false>(ch, f);
        else
            chunk_scale<false, true>(ch, f);
    }
    for (; c >= 0; c -= gridDim.x)
        if (const Chunk ch = chunks[c]; !leave(ch)) chunk_scale<true, true>(ch, f);
}

struct Range {
    uintptr_t lo, hi;
    bool written;
};
bool by_address(const Range& a, const Range& b) { return a.lo < b.lo; }

size_t elem_bytes(int dtype) { return dtype == NF4_DTYPE_BF16 ? 2 : 4; }

// The pieces of one tensor: a short head up to the first 16-byte boundary that both buffers
// share, then piece_bytes at a time; without such a boundary narrow pieces throughout.
template <typename F>
void pieces(const nf4_grad_tensor& t, size_t piece_bytes, F&& emit) {
    const size_t es = elem_bytes(t.dtype);
    const uint32_t type = t.dtype == NF4_DTYPE_BF16 ? kBf16 : 0;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.grad), b = reinterpret_cast<uintptr_t>(t.out);
    const bool wide = (a - b) % 16 == 0;
    const int64_t step = int64_t(piece_bytes / es);
    int64_t at = 0;
    auto put = [&](int64_t count, uint32_t flags) {
        emit(Chunk{static_cast<const char*>(t.grad) + at * es, static_cast<char*>(t.out) + at * es, uint32_t(count),
                   flags, 0});
        at += count;
    };
    if (wide && a % 16 != 0 && t.count > 0) put(std::min<int64_t>(t.count, int64_t((16 - a % 16) / es)), type);
    while (at < t.count) put(std::min(step, t.count - at), type | (wide ? kWide : 0));
}

size_t all_bytes(const nf4_grad_tensor* tensors, int n) {
    size_t all = 0;
    for (int i = 0; i < n; ++i) all += size_t(tensors[i].count) * elem_bytes(tensors[i].dtype);
    return all;
}

// 64 KB, or less where that would give fewer than about 1024 pieces: the 14 tensors of one 7B
// layer in bf16 (2.9 MB) take 12.4 us in 64 KB pieces, 7.6 us in 4 KB ones.
size_t piece_of(size_t all) {
    return std::min<size_t>(65536, std::max<size_t>(4096, (all / 1024 + 4095) & ~size_t(4095)));
}

int check_tensors(const char* fn, const nf4_grad_tensor* tensors, int n) {
    if (n < 0 || n > (1 << 20) || (n > 0 && !tensors))
        return fail(NF4_E_ARG, "%s: need tensors and 0 <= n <= 2^20 (got n=%d)", fn, n);
    for (int i = 0; i < n; ++i) {
        const nf4_grad_tensor& t = tensors[i];
        if (t.dtype != NF4_DTYPE_BF16 && t.dtype != NF4_DTYPE_F32)
            return fail(NF4_E_ARG, "%s: tensor %d: dtype %d is neither bf16 nor fp32", fn, i, t.dtype);
        if (t.count < 0 || t.count > (int64_t(1) << 36))
            return fail(NF4_E_SHAPE, "%s: tensor %d: count %lld outside 0..2^36", fn, i, (long long)t.count);
        if (t.count == 0) continue;
        const uintptr_t es = elem_bytes(t.dtype);
        if (!t.grad || !t.out || reinterpret_cast<uintptr_t>(t.grad) % es || reinterpret_cast<uintptr_t>(t.out) % es)
            return fail(NF4_E_ARG, "%s: tensor %d: NULL pointer or not aligned to its elements", fn, i);
    }
    return NF4_OK;
}

}  // namespace

}  // namespace nf4

struct nf4_grad_list {
    const nf4::Chunk* table;
    int n;         // pieces
    int in_place;  // every tensor's out is its grad
    int stream;    // first pieces that the caches cannot hold from one launch to the next
    std::vector<nf4::Range> memory;  // of the tensors and the table, in order of address, joined where they meet

    bool meets(const void* p, size_t bytes) const {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        const auto after = std::upper_bound(memory.begin(), memory.end(), nf4::Range{lo, lo, false}, nf4::by_address);
        return (after != memory.end() && after->lo < lo + bytes) || (after != memory.begin() && std::prev(after)->hi > lo);
    }
};

using namespace nf4;

extern "C" {

size_t nf4_grad_list_table(const nf4_grad_tensor* tensors, int n) {
    if (check_tensors("nf4_grad_list_table", tensors, n) != NF4_OK) return 0;
    const size_t piece = piece_of(all_bytes(tensors, n));
    size_t pieces_all = 1;
    for (int i = 0; i < n; ++i)
        pieces_all += size_t(tensors[i].count) * elem_bytes(tensors[i].dtype) / piece + 2;
    return pieces_all * sizeof(Chunk);
}

int nf4_grad_list_create(const nf4_grad_tensor* tensors, int n, void* table, size_t table_bytes, nf4_stream stream,
                         nf4_grad_list** out) {
    const char* fn = "nf4_grad_list_create";
    if (!out) return fail(NF4_E_ARG, "%s: out is NULL", fn);
    *out = nullptr;
    int st = check_tensors(fn, tensors, n);
    if (st != NF4_OK) return st;
    const size_t need = nf4_grad_list_table(tensors, n);
    if (!table || reinterpret_cast<uintptr_t>(table) % 256 != 0 || table_bytes < need)
        return fail(NF4_E_ARG, "%s: table must be 256-byte aligned device memory of at least %zu bytes (got %zu)", fn,
                    need, table_bytes);
    try {
        // a written range must not meet another tensor's range: the pieces run concurrently
        std::vector<Range> ranges;
        std::vector<Chunk> chunks;
        int in_place = 1;
        const size_t all = all_bytes(tensors, n), piece = piece_of(all);
        for (int i = 0; i < n; ++i) {
            const nf4_grad_tensor& t = tensors[i];
            if (t.count == 0) continue;
            const uintptr_t bytes = uintptr_t(t.count) * elem_bytes(t.dtype);
            const uintptr_t g = reinterpret_cast<uintptr_t>(t.grad), o = reinterpret_cast<uintptr_t>(t.out);
            ranges.push_back({o, o + bytes, true});
            if (g != o) {
                ranges.push_back({g, g + bytes, false});
                in_place = 0;
            }
            pieces(t, piece, [&](const Chunk& c) { chunks.push_back(c); });
        }
        std::sort(ranges.begin(), ranges.end(), by_address);
        uintptr_t written = 0, read = 0;
        for (const Range& r : ranges) {
            if (r.lo < written || (r.written && r.lo < read))
                return fail(NF4_E_ARG, "%s: a tensor's output overlaps another tensor (the same tensor twice?)", fn);
            (r.written ? written : read) = std::max(r.written ? written : read, r.hi);
        }
        if (chunks.size() * sizeof(Chunk) > table_bytes)
            return fail(NF4_E_SHAPE, "%s: %zu pieces do not fit the table", fn, chunks.size());
        const uintptr_t at = reinterpret_cast<uintptr_t>(table);
        const Range own{at, at + chunks.size() * sizeof(Chunk), false};
        for (const Range& r : ranges)
            if (r.lo < own.hi && own.lo < r.hi) return fail(NF4_E_ARG, "%s: the table overlaps a tensor", fn);
        ranges.push_back(own);
        std::sort(ranges.begin(), ranges.end(), by_address);
        std::vector<Range> memory;
        for (const Range& r : ranges) {
            if (memory.empty() || r.lo > memory.back().hi)
                memory.push_back(r);
            else
                memory.back().hi = std::max(memory.back().hi, r.hi);
        }
        if (!chunks.empty()) {
            hipStream_t s = static_cast<hipStream_t>(stream);
            hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
            if (hipStreamIsCapturing(s, &capture) != hipSuccess || capture != hipStreamCaptureStatusNone) {
                (void)hipGetLastError();
                return fail(NF4_E_STATE, "%s: a list is made before a capture, not within one", fn);
            }
            hipError_t e = hipMemcpyAsync(table, chunks.data(), chunks.size() * sizeof(Chunk), hipMemcpyHostToDevice, s);
            if (e == hipSuccess) e = hipStreamSynchronize(s);  // the source is this call's own
            if (e != hipSuccess) return fail(NF4_E_HIP, "%s: %s", fn, hipGetErrorString(e));
        }
        *out = new nf4_grad_list{static_cast<const Chunk*>(table), int(chunks.size()), in_place,
                                 double(all) > kCacheBytes ? int(double(chunks.size()) * (1.0 - kCacheBytes / double(all))) : 0,
                                 std::move(memory)};
    } catch (const std::bad_alloc&) {
        return fail(NF4_E_OOM, "%s: out of host memory", fn);
    }
    return NF4_OK;
}

int nf4_grad_list_destroy(nf4_grad_list* list) {
    if (!list) return fail(NF4_E_ARG, "nf4_grad_list_destroy: NULL list");
    delete list;
    return NF4_OK;
}

size_t nf4_grad_workspace(void) { return kMaxShares * sizeof(double); }

static int grad_run(const char* fn, const nf4_grad_list* list, float max_norm, int scale, float* norm, void* ws,
                    size_t ws_bytes, nf4_stream stream) {
    if (!list) return fail(NF4_E_ARG, "%s: NULL list", fn);
    if (!norm || reinterpret_cast<uintptr_t>(norm) % 4 != 0)
        return fail(NF4_E_ARG, "%s: norm must be 4-byte aligned and not NULL", fn);
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < nf4_grad_workspace())
        return fail(NF4_E_ARG, "%s: workspace must be 256-byte aligned and at least %zu bytes (got %zu)", fn,
                    nf4_grad_workspace(), ws_bytes);
    const ByteRange norm_at{norm, sizeof(float)}, ws_at{ws, nf4_grad_workspace()};
    if (norm_at.meets(ws_at) || list->meets(norm, norm_at.bytes) || list->meets(ws, ws_at.bytes))
        return fail(NF4_E_ARG, "%s: norm or the workspace overlaps another argument, a tensor of the list or its table", fn);
    hipStream_t s = static_cast<hipStream_t>(stream);
    double* shares = static_cast<double*>(ws);
    const int wgs = std::min(list->n, kMaxShares);
    if (wgs)
        hipLaunchKernelGGL(k_grad_norm, dim3(unsigned(wgs)), dim3(kThreads), 0, s, list->table, list->n,
                           list->stream, shares);
    hipLaunchKernelGGL(k_grad_scale, dim3(unsigned(scale && wgs ? wgs : 1)), dim3(kThreads), 0, s, list->table, list->n,
                       shares, wgs, max_norm, scale, list->in_place, list->stream, norm);
    return check_launch(fn);
}

int nf4_grad_norm(const nf4_grad_list* list, float* norm, void* ws, size_t ws_bytes, nf4_stream stream) {
    return grad_run("nf4_grad_norm", list, 0.0f, 0, norm, ws, ws_bytes, stream);
}

int nf4_grad_clip(const nf4_grad_list* list, float max_norm, float* norm, void* ws, size_t ws_bytes,
                  nf4_stream stream) {
    if (!std::isfinite(max_norm) || max_norm < 0.0f)
        return fail(NF4_E_ARG, "nf4_grad_clip: max_norm must be finite and not negative (got %g)", double(max_norm));
    return grad_run("nf4_grad_clip", list, max_norm, 1, norm, ws, ws_bytes, stream);
}

}  // extern "C"
