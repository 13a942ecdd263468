// sa_cache.cu -- writing and reading the paged INT8 key/value cache for sm_100a.
//
// A page holds one block: 64 consecutive tokens of one sequence, for every head, as INT8
// codes [page][head][64][d] with one fp32 scale for each page and head.  Token t of sequence
// b is row t % 64 of page table[b][t / 64].
//
// append: over a block's new values of one head (keys and values apart)
//     s_new = fl(max|x| / 127),  s = s_new, or max(s_old, s_new) with older tokens in the block,
//     old codes  c -> rint(fl(c * fl(s_old / s))),   new codes rint(fl(x / s)) within +-127,
// where fl is one rounding to fp32 and rint rounds ties to even; s = 0 gives codes 0.  The
// maximum is taken on the bits of |x|, so a NaN or infinity reaches the scale and the block
// reads back as NaN instead of hiding it.
//
// What bounds it: two bytes read and one written per value (68132 tokens, 16 heads of 64: 83 us,
// 5.1 TB/s; reading them back as fp32 134 us, 5.2 TB/s); for one token a sequence, the
// chain of dependent loads (sequence, page, scale).  One block of threads takes one block of
// tokens and some heads, half of it the keys, half the values; a head's values stay in
// registers between the maximum and the codes.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sa_internal.h"

namespace sa {

__device__ int g_cache_status;  // 0 = OK, 8 = an index read on the device was out of range

namespace {

constexpr int kVec = 4;    // 8-value chunks of a thread
constexpr int kWaves = 6;  // blocks of threads an SM, at least, before a block takes more heads

__device__ __forceinline__ void record_bad_index() { atomicExch(&g_cache_status, 8); }

// The block of tokens that this thread block serves.  Sequence b has the slots
// base(b) = tok_start[b] / 64 + 2 b up to base(b + 1): at least as many as its n tokens can
// touch blocks, ceil(n / 64) + 1, because the floor of a difference is at most one short.
struct Place {
    int b, ts, n, start, len, block, lo, hi;  // lo, hi: positions of the tokens in this block
    int page;
    bool first;  // the sequence's first slot
};

template <int kThreads, bool MANY>
__device__ __forceinline__ bool find_place(const CacheArgs &A, int slot, Place &P)
{
    // base is increasing in b: b is the last one whose base is at or below the slot; the thread
    // that looks at it has the rest of what there is to know already on its way.  MANY, more sequences
    // than threads: first, each round leaves those between two that the threads looked at (where every slot
    // looked through all, 65536 tokens of as many sequences took 16 ms, now 0.8; one round costs 1 % of
    // append-prompts, so fewer sequences have kernels without it).  Where offsets decrease, the count names
    // some other sequence, which finds that the slot is not its own.
    __shared__ int found[4];
    int from = 0, to = A.B;
    if constexpr (MANY) {
        while (to - from > kThreads) {
            const int step = (to - from + kThreads - 1) / kThreads, b = from + int(threadIdx.x) * step;
            const int c = __syncthreads_count(b < to && A.tok_start[b] / kPage + 2 * b <= slot);
            if (c == 0) return false;
            from += (c - 1) * step;
            to = min(to, from + step);
        }
    }
    const int b = from + int(threadIdx.x);
    int ts = 0, te_b = 0, len = 0;
    if (b < to) {
        ts = A.tok_start[b];
        te_b = A.tok_start[b + 1];
        len = A.kv_lens[b];
    }
    const int c = __syncthreads_count(b < to && ts / kPage + 2 * b <= slot);
    if (int(threadIdx.x) == c - 1) {
        found[0] = b;
        found[1] = ts;
        found[2] = te_b;
        found[3] = len;
    }
    __syncthreads();
    if (c == 0) return false;
    P.b = found[0];
    P.ts = found[1];
    const int te = found[2];
    P.len = found[3];
    P.n = te - P.ts;
    if (P.ts < 0 || te < P.ts || te > A.T || P.len < 0 || P.len > int64_t(A.max_pages) * kPage) {
        if (threadIdx.x == 0) record_bad_index();
        return false;
    }
    P.start = P.len - P.n;
    const int base = P.ts / kPage + 2 * P.b;
    P.first = slot == base;
    P.block = max(P.start, 0) / kPage + slot - base;
    if (P.n == 0) return false;
    P.lo = max(P.start, P.block * kPage);
    P.lo = max(P.lo, 0);
    P.hi = min(P.len, P.block * kPage + kPage);
    P.page = -1;
    if (P.lo >= P.hi) return P.first;  // padding tokens only
    P.page = A.table[int64_t(P.b) * A.max_pages + P.block];
    if (P.page < 0 || P.page >= A.num_pages) {
        if (threadIdx.x == 0) record_bad_index();
        P.page = -2;
    }
    return true;
}

template <typename T>
__device__ __forceinline__ float bits_to_float(uint32_t h);
template <>
__device__ __forceinline__ float bits_to_float<__nv_bfloat16>(uint32_t h)
{
    return __uint_as_float(h << 16);
}
template <>
__device__ __forceinline__ float bits_to_float<__half>(uint32_t h)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return (uint32_t(a) & 0xffu) | ((uint32_t(b) & 0xffu) << 8) | ((uint32_t(c) & 0xffu) << 16) | (uint32_t(d) << 24);
}

__device__ __forceinline__ int clamp127(float q) { return max(-127, min(127, __float2int_rn(q))); }

// Four codes rint(fl(x / s)) from the reciprocal r of s, correctly rounded: one step of Newton's
// iteration with the exact remainder, q = x r, q + (x - q s) r, gives the correctly rounded
// quotient (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) as long as nothing leaves the normal range, which the caller sees to.  Adding
// 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float r)
{
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = x[i] * r;
        y[i] = __float_as_uint(fmaf(fmaf(-q, s, x[i]), r, q) + 12582912.0f);
    }
    return __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
}

// Eight codes of eight values; reciprocals only where x, s and the quotients stay normal, or
// round to 0: s in [2^-100, 2^100].
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4 &x, float s, float r)
{
    const bool plain = s >= 7.9e-31f && s <= 1.26e30f;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const float f[4] = {bits_to_float<T>(w[2 * y] & 0xffffu), bits_to_float<T>(w[2 * y] >> 16),
                            bits_to_float<T>(w[2 * y + 1] & 0xffffu), bits_to_float<T>(w[2 * y + 1] >> 16)};
        if (plain) {
            out[y] = codes4(f, s, r);
        } else {
            int c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = s == 0.0f ? 0 : clamp127(__fdiv_rn(f[k], s));
            out[y] = pack4(c[0], c[1], c[2], c[3]);
        }
    }
    return make_uint2(out[0], out[1]);
}

// Eight older codes by the ratio r of the scales.
__device__ __forceinline__ void rescale8(int8_t *codes, float r)
{
    uint2 *p = reinterpret_cast<uint2 *>(codes);
    const uint2 w = *p;
    int c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int code = int(int8_t((k < 4 ? w.x : w.y) >> (8 * (k & 3))));
        c[k] = clamp127(__fmul_rn(float(code), r));
    }
    *p = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// The block's scale from the bits of its largest new |x|, and the old one if there are older tokens.
template <typename T>
__device__ __forceinline__ float new_scale(uint32_t bits, float s_old, bool older)
{
    const float s_new = __fdiv_rn(bits_to_float<T>(bits), 127.0f);
    return !older || s_new > s_old || s_new != s_new ? s_new : s_old;
}

template <typename T, int D, bool MANY>
__global__ void __launch_bounds__(4 * D, 1024 / (4 * D)) cache_append_kernel(const CacheArgs A)
{
    constexpr int kThreads = 4 * D, kHalf = kThreads / 2;
    constexpr int kChunks = D / 8;  // 8-value chunks of a row
    static_assert(kVec * kHalf == kPage * kChunks, "a block's chunks");
    __shared__ uint32_t most[2][kThreads / 32];
    chain_begin();
    Place P;
    if (!find_place<kThreads, MANY>(A, int(blockIdx.x) / A.head_cuts, P) || P.page < 0) return;
    const int side = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    const int h_lo = int(blockIdx.x) % A.head_cuts * A.heads_per_block, h_hi = min(A.H, h_lo + A.heads_per_block);
    const int row_lo = P.lo - P.block * kPage, row_hi = P.hi - P.block * kPage;  // new rows
    const int64_t stride = side ? A.v_stride : A.k_stride;
    const T *src = static_cast<const T *>(side ? A.v : A.k) + (P.ts + int64_t(P.block * kPage - P.start)) * stride;
    int8_t *codes = (side ? A.v_codes : A.k_codes) + int64_t(P.page) * A.H * (kPage * D);
    float *scale = (side ? A.v_scale : A.k_scale) + int64_t(P.page) * A.H;

    for (int head = h_lo; head < h_hi; ++head) {
        uint4 x[kVec];
        uint32_t top = 0;  // two 16-bit maxima of |x|'s bits
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = tid + i * kHalf, row = v / kChunks, c = v % kChunks;
            x[i] = make_uint4(0, 0, 0, 0);
            if (row >= row_lo && row < row_hi)
                x[i] = *reinterpret_cast<const uint4 *>(src + row * stride + head * D + 8 * c);
        }
        const float s_old = row_lo > 0 ? scale[head] : 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        uint32_t *turn = most[head & 1];
        if ((threadIdx.x & 31) == 0) turn[threadIdx.x / 32] = top;
        __syncthreads();
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kHalf / 32; ++i) m = max(m, turn[side * (kHalf / 32) + i]);
        const float s = new_scale<T>(m, s_old, row_lo > 0);
        int8_t *cell = codes + int64_t(head) * (kPage * D);
        if (row_lo > 0 && !(s == s_old)) {
            const float r = __fdiv_rn(s_old, s);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = tid + i * kHalf;
                if (v / kChunks < row_lo) rescale8(cell + 8 * v, r);
            }
        }
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = tid + i * kHalf, row = v / kChunks;
            if (row >= row_lo && row < row_hi) *reinterpret_cast<uint2 *>(cell + 8 * v) = codes8<T>(x[i], s, r);
        }
        if (tid == 0) scale[head] = s;
    }
}

// The same for few new tokens a sequence: a warp takes one head's keys or values alone, so that
// nothing waits for threads that have no value, and reads the values again if they are more rows
// than it holds.  64 sequences of one token, 8 heads of 128: 3.5 us instead of 9.5.
constexpr int kFewTokens = 4, kFewWarps = 8;
template <typename T, int D, bool MANY>
__global__ void __launch_bounds__(32 * kFewWarps) cache_append_few_kernel(const CacheArgs A)
{
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows at once
    chain_begin();
    Place P;
    if (!find_place<32 * kFewWarps, MANY>(A, int(blockIdx.x) / A.head_cuts, P) || P.page < 0) return;
    const int lane = threadIdx.x & 31, unit = int(blockIdx.x) % A.head_cuts * kFewWarps + int(threadIdx.x >> 5);
    const int head = unit / 2, side = unit % 2;
    if (head >= A.H) return;
    const int row_lo = P.lo - P.block * kPage, row_hi = P.hi - P.block * kPage;  // new rows
    const int64_t stride = side ? A.v_stride : A.k_stride, cell = int64_t(P.page) * A.H + head;
    const T *src = static_cast<const T *>(side ? A.v : A.k) + (P.ts + int64_t(P.block * kPage - P.start)) * stride + head * D;
    int8_t *codes = (side ? A.v_codes : A.k_codes) + cell * (kPage * D);
    float *scale = (side ? A.v_scale : A.k_scale) + cell;
    auto load = [&](int row) {
        return row < row_hi ? *reinterpret_cast<const uint4 *>(src + row * stride + 8 * (lane % kLanes)) : make_uint4(0, 0, 0, 0);
    };
    const int row0 = row_lo + lane / kLanes;
    uint4 x = load(row0);
    const float s_old = row_lo > 0 ? *scale : 0.0f;
    uint32_t top = 0;
    for (int row = row0;;) {
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                     __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        if ((row += kRows) >= row_hi) break;
        x = load(row);
    }
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    const float s = new_scale<T>(m, s_old, row_lo > 0);
    if (row_lo > 0 && !(s == s_old)) {
        const float r = __fdiv_rn(s_old, s);
        for (int v = lane; v < row_lo * kLanes; v += 32) rescale8(codes + 8 * v, r);
    }
    const float r = __frcp_rn(s);
    if (row_hi - row_lo > kRows) x = load(row0);
    for (int row = row0; row < row_hi; row += kRows) {
        if (row > row0) x = load(row);
        *reinterpret_cast<uint2 *>(codes + row * D + 8 * (lane % kLanes)) = codes8<T>(x, s, r);
    }
    if (lane == 0) *scale = s;
}

// 16 bytes of output
template <typename T>
__device__ __forceinline__ void store16(T *p, const float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void store16<float>(float *p, const float (&f)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16 *p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store16<__half>(__half *p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// N codes from p on as floats
template <int N>
__device__ __forceinline__ void load_codes(const int8_t *p, float (&f)[N])
{
    if constexpr (N == 8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = float(int8_t((k < 4 ? w.x : w.y) >> (8 * (k & 3))));
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = float(int8_t(w >> (8 * k)));
    }
}

// Writes are most of it, so a thread takes as many codes as fill 16 bytes of the output.
constexpr int kReadThreads = 256;
template <typename T, int D, bool MANY>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheArgs A)
{
    constexpr int kThreads = kReadThreads, kHalf = kThreads / 2, kCodes = 16 / int(sizeof(T)), kChunks = D / kCodes;
    constexpr int kPer = kPage * kChunks / kHalf;
    chain_begin();
    Place P;
    if (!find_place<kThreads, MANY>(A, int(blockIdx.x) / A.H, P)) return;
    const int head = int(blockIdx.x) % A.H, side = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    T *dst = static_cast<T *>(const_cast<void *>(side ? A.v : A.k));
    if (!dst) return;
    const int64_t stride = int64_t(A.H) * D;
    if (P.first && P.start < 0) {  // positions before the sequence: zero
        const float zero[kCodes] = {};
        for (int64_t i = tid; i < int64_t(min(-P.start, P.n)) * kChunks; i += kHalf)
            store16<T>(dst + (P.ts + i / kChunks) * stride + head * D + kCodes * (i % kChunks), zero);
    }
    if (P.lo >= P.hi) return;
    const int64_t cell = int64_t(max(P.page, 0)) * A.H + head;
    const int8_t *codes = (side ? A.v_codes : A.k_codes) + cell * (kPage * D);
    const float s = P.page < 0 ? __int_as_float(0x7fffffff) : (side ? A.v_scale : A.k_scale)[cell];
    const int row_lo = P.lo - P.block * kPage, row_hi = P.hi - P.block * kPage;
    dst += (P.ts + int64_t(P.block * kPage - P.start)) * stride + head * D;
#pragma unroll 8
    for (int i = 0; i < kPer; ++i) {
        const int v = tid + i * kHalf, row = v / kChunks, c = v % kChunks;
        if (row < row_lo || row >= row_hi) continue;
        float f[kCodes];
        load_codes(codes + kCodes * v, f);
#pragma unroll
        for (int k = 0; k < kCodes; ++k) f[k] *= s;
        store16<T>(dst + row * stride + kCodes * c, f);
    }
}

// Neighbouring blocks take the heads of the same tokens, whose memory is contiguous.
int64_t slots_of(const CacheArgs &a) { return a.T / kPage + 2 * int64_t(a.B); }

template <typename T, int D>
cudaError_t append_for(CacheArgs a, cudaStream_t st)
{
    if (a.T <= int64_t(kFewTokens) * a.B) {
        a.head_cuts = int(cdiv(2 * int64_t(a.H), kFewWarps));
        return launch_chained(a.B > 32 * kFewWarps ? cache_append_few_kernel<T, D, true> : cache_append_few_kernel<T, D, false>,
                              dim3(unsigned(slots_of(a) * a.head_cuts)), 32 * kFewWarps, 0, st, a);
    }
    // several heads a block where there are blocks enough to fill the SMs several times over
    const int64_t blocks = (a.T / kPage + a.B) * int64_t(a.H);  // about so many are not empty
    a.heads_per_block = int(std::max<int64_t>(1, std::min<int64_t>(8, blocks / (kWaves * std::max(1, device_sms())))));
    a.head_cuts = int(cdiv(a.H, a.heads_per_block));
    const int64_t grid = slots_of(a) * a.head_cuts;
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    return launch_chained(a.B > 4 * D ? cache_append_kernel<T, D, true> : cache_append_kernel<T, D, false>, dim3(unsigned(grid)),
                          4 * D, 0, st, a);
}

template <typename T, int D>
cudaError_t read_for(const CacheArgs &a, cudaStream_t st)
{
    const int64_t grid = slots_of(a) * a.H;
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    return launch_chained(a.B > kReadThreads ? cache_read_kernel<T, D, true> : cache_read_kernel<T, D, false>,
                          dim3(unsigned(grid)), kReadThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs &a, int dtype, cudaStream_t st)
{
    if (dtype == 0) return a.d == 128 ? append_for<__nv_bfloat16, 128>(a, st) : append_for<__nv_bfloat16, 64>(a, st);
    return a.d == 128 ? append_for<__half, 128>(a, st) : append_for<__half, 64>(a, st);
}

cudaError_t launch_cache_read(const CacheArgs &a, int dtype, cudaStream_t st)
{
    if (dtype == 0) return a.d == 128 ? read_for<__nv_bfloat16, 128>(a, st) : read_for<__nv_bfloat16, 64>(a, st);
    if (dtype == 1) return a.d == 128 ? read_for<__half, 128>(a, st) : read_for<__half, 64>(a, st);
    return a.d == 128 ? read_for<float, 128>(a, st) : read_for<float, 64>(a, st);
}

cudaError_t read_and_clear_cache_status(int *status)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(status, g_cache_status, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_cache_status, &zero, sizeof(int));
}

}  // namespace sa
