// sa_cache_attn.cuh -- what the two attention kernels over the paged INT8 cache share: codes to
// fp16, query rows to fp16, the sequences' arrays, outputs.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sa_internal.h"
#include "sa_ptx.cuh"

namespace sa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }

// two of four bytes u = code + 128 to fp16: 0x6400 + u is 1024 + u, less 1152 is the code
__device__ __forceinline__ uint32_t bytes_to_h2(uint32_t u, uint32_t sel)
{
    const uint32_t p = __byte_perm(u, 0x64646464u, sel);
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    return h2(__hsub2(*reinterpret_cast<const __half2 *>(&p), bias));
}

__device__ __forceinline__ uint32_t pack_out(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_out(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// four consecutive values of a row as floats
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&f)[4])
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const __half *p, float (&f)[4])
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// First token, tokens and cached length of sequence b; false (and an empty sequence) if they
// are out of range.
__device__ __forceinline__ bool load_span(const CacheAttnArgs &A, int b, int &ts, int &n, int &len)
{
    ts = A.tok_start[b];
    const int te = A.tok_start[b + 1];
    len = A.kv_lens[b];
    n = te - ts;
    if (ts >= 0 && te >= ts && te <= A.T && len >= 0 && len <= int64_t(A.max_pages) * kPage) return true;
    ts = n = len = 0;
    return false;
}

// The tensor-core kernel's work: a segment is kRowsSeg rows (query token and shared head) of a
// sequence, a step two blocks of keys.  Segment p of the n new tokens of a sequence with len cached
// ones, G query heads on each head, sees the blocks [blo, bhi), at least one step.
constexpr int kRowsSeg = 256;
struct Reach {
    int blo, bhi;
    __host__ __device__ int steps() const { return bhi - blo > 2 ? (bhi - blo + 1) / 2 : 1; }
};
__host__ __device__ __forceinline__ Reach reach_of(int n, int len, int G, int causal, int window, int p)
{
    const int rows = n * G, pos0 = len - n, end = p * kRowsSeg + kRowsSeg;
    const int i_lo = p * kRowsSeg / G, i_hi = ((rows < end ? rows : end) - 1) / G;
    const int last = causal || pos0 + i_hi < 0 ? pos0 + i_hi : len - 1;
    const int seen = pos0 + i_lo - window + 1, first = window > 0 && seen > 0 ? seen : 0;
    Reach r;
    r.blo = first / kPage;
    r.bhi = last < first ? r.blo : last / kPage + 1;
    return r;
}
// Steps of its segments p0, p0 + stride, ...: 2^22 segments of 2^23 steps are accepted, so 64 bits.
__host__ __device__ __forceinline__ int64_t steps_of(int n, int len, int G, int causal, int window, int p0, int stride)
{
    int64_t sum = 0;
    for (int p = p0; p < (n * G + kRowsSeg - 1) / kRowsSeg; p += stride) sum += reach_of(n, len, G, causal, window, p).steps();
    return sum;
}

// log2 of a value scale: -inf for 0, NaN for one that is not finite (its block reads as NaN).
__device__ __forceinline__ float log2_scale(float s) { return s < INFINITY ? log2f(s) : __int_as_float(0x7fffffff); }

// Weights are 2^(x + log2 scale_v + bits - w) while they are summed, relative to 2^m when the sums are
// written: f * power = 2^(w - m - bits), in two factors where one would leave the normal range (value
// scales below about 2^-100).  The sums are 0 where w = -inf (no scale above 0).
__device__ __forceinline__ void power_of(float w, float m, float bits, float &f, float &power)
{
    const float k = w == -INFINITY ? 0.0f : w - m - bits, near = fminf(fmaxf(k, -100.0f), 100.0f);
    f = ex2_approx(k - near);
    power = ex2_approx(near);
}
// A step's sum of p is taken from the weights as long as the one at x = m is 2^-90 or more, so that
// those 2^-30 of it are still normal.
constexpr float kAtLeast = -90.0f;

// The power of two, and its inverse, that brings a row whose largest magnitude is `top` to
// [1, 4): bf16 has more range than fp16.  Values that leave fp16's normal range then are below
// 2^-14 of the row's largest; all others stay exact.
__device__ __forceinline__ void row_power(float top, float &up, float &down)
{
    int ex = int(__float_as_uint(top) >> 23) - 127;
    ex = (top == 0.0f || ex == 128) ? 0 : max(-126, min(126, ex));
    up = __uint_as_float(uint32_t(127 - ex) << 23);
    down = __uint_as_float(uint32_t(127 + ex) << 23);
}

}  // namespace sa
