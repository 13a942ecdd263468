// sa_rope.cu -- rotary positions of queries and keys for sm_100a.
//
// Pair i of a head's first `rot` channels, (a, b) = channels (i, i + rot/2) or, interleaved,
// (2i, 2i + 1), becomes amplitude * (a cos f - b sin f, b cos f + a sin f) with
// f = pos[axis of i] * freqs[i]; the other channels are copied.  `inverse` turns by -f, which
// is the transposed map (and so the gradient's).
//
// Angles: the product is taken in fp64 in units of whole turns and reduced by the nearest
// integer there, so a position of 2^20 loses nothing; sincospif then works on [-1, 1].
//
// What bounds it: reading and writing each value once (32760 tokens, 12 + 12 heads of 128 in bf16:
// 71 us, 5.7 TB/s).  The sines of a token serve all its
// heads, so a block takes a few tokens of all heads (or a slice of the heads where there are
// few tokens), puts the sines in shared memory once, and each thread keeps the eight pairs it
// needs in registers while it walks the heads.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kTileUnits = 64;  // (token, 16-channel unit) pairs of a block's tile

// eight consecutive values as floats, and back with one rounding
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ void get(float (&f)[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ static void store(float *p, const float (&f)[8])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <typename T, typename T2>
struct Vec8Half {
    uint4 v;
    __device__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
};
template <>
struct Vec8<__nv_bfloat16> : Vec8Half<__nv_bfloat16, __nv_bfloat162> {
    __device__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static void store(__nv_bfloat16 *p, const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec8<__half> : Vec8Half<__half, __half2> {
    __device__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    __device__ static void store(__half *p, const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs A)
{
    __shared__ float2 table[kTileUnits * 8];  // [token of the tile][pair]
    chain_begin();
    const int units = A.d / 16, tile_tokens = A.tile_tokens, half = A.rot / 2;
    const int tiles = (A.N + tile_tokens - 1) / tile_tokens;
    const int64_t b = blockIdx.x / tiles;
    const int n0 = int(blockIdx.x % tiles) * tile_tokens;
    const int ntok = min(tile_tokens, A.N - n0);

    const int tu = tile_tokens * units, slots = kThreads / tu;
    const int slot = threadIdx.x / tu, rest = threadIdx.x - slot * tu;
    const int t = rest / units, u = rest - t * units;
    const bool active = slot < slots && t < ntok;
    // The thread's two chunks of 8 channels, each contiguous from thread to thread: the two halves of
    // eight pairs, or (interleaved, and channels that do not turn) four pairs each.
    const bool pairs = !INTERLEAVED && 16 * u < A.rot;
    const int c0 = INTERLEAVED || pairs ? 8 * u : 8 * u + half;
    const int c1 = INTERLEAVED ? A.d / 2 + 8 * u : pairs ? half + 8 * u : c0 + (A.d - A.rot) / 2;
    const bool turned0 = INTERLEAVED ? c0 < A.rot : pairs, turned1 = INTERLEAVED ? c1 < A.rot : pairs;
    const int heads = A.io[0].heads + A.io[1].heads;
    const int h_end = min(heads, int(blockIdx.y + 1) * A.heads_per_block);
    int h0 = blockIdx.y * A.heads_per_block + slot;

    constexpr int kUnroll = 2;  // more in flight costs blocks on an SM: 4 takes 81 us for 403 MB, 2 72, 1 74
    Vec8<T> lo[kUnroll], hi[kUnroll];
    T *dst[kUnroll];
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int h = h0 + k * slots;
            dst[k] = nullptr;
            if (!active || h >= h_end) continue;
            const bool second = h >= A.io[0].heads;
            const RopeIo &io = A.io[second ? 1 : 0];
            const int64_t hh = second ? h - A.io[0].heads : h, n = n0 + t;
            const T *src = static_cast<const T *>(io.x) + b * io.xb + hh * io.xh + n * io.xn;
            T *out = static_cast<T *>(io.y) + b * io.yb + hh * io.yh + n * io.yn;
            if (!turned0 && !turned1 && src == out) continue;  // in place: nothing to copy
            dst[k] = out;
            lo[k].load(src + c0);
            hi[k].load(src + c1);
        }
    };
    load();  // on their way while the sines are found

    for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
        const int ti = i / half, p = i - ti * half;
        const int axis = (p >= A.axis_end[0]) + (p >= A.axis_end[1]) + (p >= A.axis_end[2]);
        const int pos = A.pos[axis * A.pos_axis_stride + b * A.pos_batch_stride + n0 + ti];
        // whole turns drop out: 0.15915... = 1 / (2 pi)
        const double turns = double(pos) * (A.freqs[p] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * float(turns - rint(turns)), &s, &c);
        table[i] = make_float2(c * A.amplitude, s * (A.inverse ? -A.amplitude : A.amplitude));
    }
    __syncthreads();
    if (!active) return;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int p = INTERLEAVED ? ((i < 4 ? c0 : c1) / 2 + (i & 3)) : c0 + i;
        const float2 w = (i < 4 ? turned0 : turned1) ? table[t * half + p] : make_float2(1.0f, 0.0f);
        cs[i] = w.x;
        sn[i] = w.y;
    }
    while (true) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (!dst[k]) continue;
            float x[8], y[8];
            lo[k].get(x);
            hi[k].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!(i < 4 ? turned0 : turned1)) continue;
                float &p = INTERLEAVED ? (i < 4 ? x[2 * i & 7] : y[2 * i & 7]) : x[i];
                float &q = INTERLEAVED ? (i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7]) : y[i];
                const float a = p, e = q;
                p = a * cs[i] - e * sn[i];
                q = e * cs[i] + a * sn[i];
            }
            Vec8<T>::store(dst[k] + c0, x);
            Vec8<T>::store(dst[k] + c1, y);
        }
        h0 += kUnroll * slots;
        if (h0 >= h_end) break;
        load();
    }
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int dtype, cudaStream_t st)
{
    const int sms = device_sms();
    const int units = a.d / 16, heads = a.io[0].heads + a.io[1].heads;
    a.tile_tokens = units <= 8 ? 8 : kTileUnits / units;
    const int slots = kThreads / (a.tile_tokens * units);
    const int64_t tiles = int64_t(a.B) * cdiv(a.N, a.tile_tokens);
    // All heads of a tile in one block share its sines; with few tiles the heads are cut until
    // the blocks cover the SMs twice or a thread has one head.
    int64_t cuts = 1;
    while (tiles * cuts < 2 * sms && cdiv(heads, cuts) > slots) ++cuts;
    a.heads_per_block = int(cdiv(heads, cuts));
    const dim3 grid(unsigned(tiles), unsigned(cdiv(heads, a.heads_per_block)));
    auto go = [&](void (*kernel)(RopeArgs)) { return launch_chained(kernel, grid, kThreads, 0, st, a); };
    if (dtype == 0) return go(a.interleaved ? rope_kernel<__nv_bfloat16, true> : rope_kernel<__nv_bfloat16, false>);
    if (dtype == 1) return go(a.interleaved ? rope_kernel<__half, true> : rope_kernel<__half, false>);
    return go(a.interleaved ? rope_kernel<float, true> : rope_kernel<float, false>);
}

}  // namespace sa
