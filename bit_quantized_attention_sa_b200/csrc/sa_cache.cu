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
// What bounds it: two bytes read and one written per value; for one token a sequence, the
// chain of dependent loads (sequence, length, page, scale).  One block of threads takes one
// (block of tokens, head): half of it the keys, half the values, which stay in registers
// between the maximum and the codes.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sa_internal.h"

namespace sa {

__device__ int g_cache_status;  // 0 = OK, 8 = an index read on the device was out of range

namespace {

constexpr int kThreads = 256;
constexpr int kHalf = kThreads / 2;

__device__ __forceinline__ void record_bad_index() { atomicExch(&g_cache_status, 8); }

// The block of tokens that this thread block serves.  Sequence b has the slots
// base(b) = tok_start[b] / 64 + 2 b up to base(b + 1): at least as many as its n tokens can
// touch blocks, ceil(n / 64) + 1, because the floor of a difference is at most one short.
struct Place {
    int b, ts, n, start, len, block, lo, hi;  // lo, hi: positions of the tokens in this block
    int page;
    bool first;  // the sequence's first slot
};

__device__ __forceinline__ bool find_place(const CacheArgs &A, int slot, Place &P)
{
    // base is increasing in b: b is the number of bases at or below the slot, less one
    int below = 0;
    for (int i = 0; i < A.B; i += kThreads) {
        const int b = i + int(threadIdx.x);
        const int c = __syncthreads_count(b < A.B && A.tok_start[b] / kPage + 2 * b <= slot);
        below += c;
        if (c < kThreads) break;
    }
    P.b = below - 1;
    if (P.b < 0) return false;
    P.ts = A.tok_start[P.b];
    const int te = A.tok_start[P.b + 1];
    P.len = A.kv_lens[P.b];
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheArgs A)
{
    constexpr int kChunks = D / 8;             // 8-value chunks of a row
    constexpr int kVec = kPage * kChunks / kHalf;  // chunks of a thread
    __shared__ uint32_t most[kThreads / 32];
    Place P;
    if (!find_place(A, blockIdx.x, P) || P.page < 0) return;
    const int head = blockIdx.y, side = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    const T *src = static_cast<const T *>(side ? A.v : A.k);
    const int64_t stride = side ? A.v_stride : A.k_stride;
    const int64_t cell = int64_t(P.page) * A.H + head;
    int8_t *codes = (side ? A.v_codes : A.k_codes) + cell * (kPage * D);
    float *scale = (side ? A.v_scale : A.k_scale) + cell;
    const int row_lo = P.lo - P.block * kPage, row_hi = P.hi - P.block * kPage;  // new rows
    const float s_old = row_lo > 0 ? *scale : 0.0f;

    uint4 x[kVec];
    uint32_t top = 0;  // two 16-bit maxima of |x|'s bits
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * kHalf, row = v / kChunks, c = v % kChunks;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row >= row_lo && row < row_hi) {
            const int64_t t = P.ts + (P.block * kPage + row - P.start);
            x[i] = *reinterpret_cast<const uint4 *>(src + t * stride + head * D + 8 * c);
        }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
    }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x / 32] = top;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) m = max(m, most[side * (kHalf / 32) + i]);
    const float s_new = __fdiv_rn(bits_to_float<T>(m), 127.0f);
    const float s = (row_lo == 0 || s_new > s_old || s_new != s_new) ? s_new : s_old;

    if (row_lo > 0 && !(s == s_old)) {
        const float r = __fdiv_rn(s_old, s);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = tid + i * kHalf;
            if (v / kChunks >= row_lo) continue;
            uint2 *p = reinterpret_cast<uint2 *>(codes + 8 * v);
            const uint2 w = *p;
            int c[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int code = int(int8_t((k < 4 ? w.x : w.y) >> (8 * (k & 3))));
                c[k] = clamp127(__fmul_rn(float(code), r));
            }
            *p = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
        }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * kHalf, row = v / kChunks;
        if (row < row_lo || row >= row_hi) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        int c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = bits_to_float<T>((w[k / 2] >> (16 * (k & 1))) & 0xffffu);
            c[k] = s == 0.0f ? 0 : clamp127(__fdiv_rn(f, s));
        }
        *reinterpret_cast<uint2 *>(codes + 8 * v) =
            make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
    }
    if (tid == 0) *scale = s;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float (&f)[8])
{
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float (&f)[8])
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
__device__ __forceinline__ void store8<__half>(__half *p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs A)
{
    constexpr int kChunks = D / 8;
    constexpr int kVec = kPage * kChunks / kHalf;
    Place P;
    if (!find_place(A, blockIdx.x, P)) return;
    const int head = blockIdx.y, side = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    T *dst = static_cast<T *>(const_cast<void *>(side ? A.v : A.k));
    if (!dst) return;
    const int64_t stride = int64_t(A.H) * D;
    if (P.first && P.start < 0) {  // positions before the sequence: zero
        const float zero[8] = {};
        for (int i = tid; i < min(-P.start, P.n) * kChunks; i += kHalf)
            store8<T>(dst + (P.ts + int64_t(i / kChunks)) * stride + head * D + 8 * (i % kChunks), zero);
    }
    if (P.lo >= P.hi) return;
    const int64_t cell = int64_t(max(P.page, 0)) * A.H + head;
    const int8_t *codes = (side ? A.v_codes : A.k_codes) + cell * (kPage * D);
    const float s = P.page < 0 ? __int_as_float(0x7fffffff) : (side ? A.v_scale : A.k_scale)[cell];
    const int row_lo = P.lo - P.block * kPage, row_hi = P.hi - P.block * kPage;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * kHalf, row = v / kChunks, c = v % kChunks;
        if (row < row_lo || row >= row_hi) continue;
        const uint2 w = *reinterpret_cast<const uint2 *>(codes + 8 * v);
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = float(int8_t((k < 4 ? w.x : w.y) >> (8 * (k & 3)))) * s;
        const int64_t t = P.ts + (P.block * kPage + row - P.start);
        store8<T>(dst + t * stride + head * D + 8 * c, f);
    }
}

template <typename T>
cudaError_t append_for(const CacheArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.d == 128)
        cache_append_kernel<T, 128><<<grid, kThreads, 0, st>>>(a);
    else
        cache_append_kernel<T, 64><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_for(const CacheArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.d == 128)
        cache_read_kernel<T, 128><<<grid, kThreads, 0, st>>>(a);
    else
        cache_read_kernel<T, 64><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

dim3 place_grid(const CacheArgs &a) { return dim3(unsigned(a.T / kPage + 2 * a.B), unsigned(a.H)); }

}  // namespace

cudaError_t launch_cache_append(const CacheArgs &a, int dtype, cudaStream_t st)
{
    return dtype == 0 ? append_for<__nv_bfloat16>(a, place_grid(a), st) : append_for<__half>(a, place_grid(a), st);
}

cudaError_t launch_cache_read(const CacheArgs &a, int dtype, cudaStream_t st)
{
    if (dtype == 0) return read_for<__nv_bfloat16>(a, place_grid(a), st);
    if (dtype == 1) return read_for<__half>(a, place_grid(a), st);
    return read_for<float>(a, place_grid(a), st);
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
