// sa_cache_attn.cu -- attention of few query rows over the paged INT8 cache for sm_100a.
//
// Rows of a (sequence, key/value head) are its query tokens times the query heads that share
// the head, token-major; a tile is 8 rows, the N of one mma (the codes are its M, so that few
// rows waste little), and a warp works on one or two tiles.  For every 64-token block j
//     S = q . k8,   x = S * (scale_k[j] * sm_scale),   p = exp(x - m),
//     acc = acc * alpha + (p * scale_v[j]) . v8,   l = l * alpha + sum p,
// with m, l and acc in fp32; in the end o = acc / l and lse = m + log l.
//
// The codes are exact in fp16, and so is q after a power of two for each row (its exponent goes
// into the row's score scale), so S has no rounding before its fp32 accumulator.  P, rounded to
// fp16, is 2^15 * p * scale_v[j] / 2^w, both powers of two in the exponent (in powers of two,
// x + log2 scale_v[j] - w): w, a whole number, is the row's largest such sum so far, rounded up.  So P
// is at most 2^15, its relative error 2^-11, and what is below 2^-29 of the row's largest product of
// weight and scale falls to fp16's subnormals.  w is over the keys that the row sees: no block that it
// does not see, and no other row of the tile, changes it.  acc is kept in units of 2^(w - 15); the sum of
// p, relative to 2^m with m rounded up, is the sum of P before its rounding times a power of two.
//
// What bounds it: reading 2 d bytes for each cached token and head.  Measured, 4 sequences of
// 70001 to 131072 tokens, 32 query heads on 8 of 128: 157 us for 900 MB, 5.7 TB/s (a plain copy
// has 6.55), and 10 for the joining, some of it hidden.  So every warp is a worker
// of its own with a ring of TMA tiles in shared memory (K and V of a block are 64 x d bytes
// each), and the blocks of all (sequence, head, tile) segments, laid out one after another, are
// cut into equal ranges, one for each worker, whatever the lengths.  A range may begin or end
// inside a segment: such pieces go to the workspace as (acc, m, l) and combine_kernel joins
// them in the order of the workers, so results do not depend on timing.
//
// The tiles arrive with TMA's 128-byte swizzle (16-byte chunk c of the 128-byte line r at
// c ^ (r & 7)), which makes the 16-byte reads below free of bank conflicts at d = 128: the
// contraction index of an mma may be permuted freely as long as both operands agree, and so
// may the keys of a tile (scores and values) and the channels (columns of acc).
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sa_cache_attn.cuh"
#include "sa_internal.h"
#include "sa_ptx.cuh"

namespace sa {

__device__ int g_cache_attn_status;  // 0 = OK, 6 = a bounded wait expired, 8 = bad index

namespace {

// Rows of a sequence and head, on average, up to which this kernel takes a call; the others go to
// the tensor-core kernel of sa_cache_chunk.cu.  Measured at d = 128, 8 heads (this kernel / that
// one, us): 16 rows, 16 sequences of 4000 tokens 50 / 70, 64 of them 140 / 234, one of 60000
// 70 / 76; 24 rows, which are read twice here: 78 / 71, 252 / 237, 85 / 77.  The average is all
// that the host knows (lengths are on the device), so a long piece among single tokens stays here, each
// of its tiles reading the sequence's blocks: 255 single tokens and 2000 over 8000 728 us, as two calls
// 199 and 81; 63 and 500 over 4000 153, as two calls 65 and 41.
constexpr int kFewRows = 16;
constexpr float kPBits = 15.0f;
// Blocks of one worker, two tiles each, are counted in 32 bits; a call of more (minutes of work) is left out.
constexpr int64_t kMaxChunk = 1 << 29;

// D: head size; NT: tiles of eight rows that a warp works on at once.  One tile leaves registers
// for twelve warps, with a ring of two slots (a K or V tile of 64 x D bytes each); two tiles for
// eight warps with three.
template <int D, int NT>
struct Sizes {
    static constexpr int kRows = 8 * NT;
    static constexpr int kWarps = NT == 1 ? 12 : 8, kThreads = 32 * kWarps;
    static constexpr int kSlots = NT == 1 ? 2 : 3;
    static constexpr uint32_t kTile = 64 * D;
    static constexpr uint32_t kOffBar = kWarps * kSlots * kTile;
    static constexpr uint32_t kBytes = kOffBar + kWarps * kSlots * 8;
    static constexpr uint32_t kAlloc = kBytes + 1024;
    static constexpr int kPart = kRows * (D + 2);  // floats of a partial result
};
static_assert(Sizes<128, 1>::kAlloc <= 220 * 1024 && Sizes<128, 2>::kAlloc <= 220 * 1024, "shared memory per CTA");
constexpr int kMaxWarps = 12;

__device__ __forceinline__ void record(int what) { atomicMax(&g_cache_attn_status, what); }

// A sequence as the kernels see it: `tiles` tiles of its rows for each head, `nb` blocks for
// each tile, from block `lo` on.  Every segment has a block at least, so that some worker
// writes its rows; blocks that a tile sees nothing of are passed over.
struct Seq {
    int ts, n, len, tiles, lo, nb;
    __device__ int64_t blocks(int heads) const { return int64_t(heads) * tiles * nb; }
};

__device__ __forceinline__ Seq load_seq(const CacheAttnArgs &A, int b, int rows)
{
    Seq s;
    if (!load_span(A, b, s.ts, s.n, s.len)) record(8);
    s.tiles = (s.n * A.G + rows - 1) / rows;
    s.lo = A.window > 0 ? max(0, s.len - s.n - A.window + 1) / kPage : 0;
    s.nb = max(1, (s.len + kPage - 1) / kPage - s.lo);
    return s;
}

// An 8 x 8 matrix of 16-bit values, two of a row in each lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One block of the flattened work, held by one lane of a worker's window of 32.
struct Entry {
    int b, seg, blk;   // sequence, head * tiles + tile, block of the sequence (absolute)
    int line;          // first 128-byte line of its tiles in the cache
    float sk, lg;      // scale_k and log2 scale_v
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Sizes<D, NT>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CacheAttnArgs A)
{
    using S = Sizes<D, NT>;
    constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kSlots = S::kSlots, kRows = S::kRows;
    constexpr int kSteps = D / 16;   // k16 steps of k8 . q
    constexpr int kQuads = D / 64;   // 16-byte chunks of a key row that a lane reads
    constexpr int kMT = D / 16;      // 16-channel tiles of acc
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int64_t prefix[kThreads + 1];
    __shared__ int64_t warp_sum[kWarps];
    __shared__ int abort_word[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;

    chain_begin();
    // ---- the flattened work: thread t sums the sequences [t * per, (t + 1) * per)
    const int per = (A.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = int(threadIdx.x) * per + i;
        if (b < A.B) mine += load_seq(A, b, S::kRows).blocks(A.H);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    uint8_t *ring = smem + warp * kSlots * S::kTile;
    const uint32_t ring_addr = smem_u32(ring);
    const uint32_t bars = smem_u32(smem) + S::kOffBar + uint32_t(warp * kSlots) * 8;
    volatile int *abort_flag = &abort_word[warp];
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(bars + 8 * i, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    prefix[threadIdx.x] = before + incl - mine;
    if (threadIdx.x == kThreads - 1) {
        const bool fits = before + incl <= kMaxChunk * kWarps * int64_t(gridDim.x);
        if (!fits) record(8);
        prefix[kThreads] = fits ? before + incl : 0;
    }
    __syncthreads();
    const int64_t total = prefix[kThreads];

    // ---- this worker's range [w * chunk, end)
    const int workers = int(gridDim.x) * kWarps;
    const int w = warp * int(gridDim.x) + int(blockIdx.x);
    const int64_t chunk = (total + workers - 1) / workers;
    const int64_t start = w * chunk;
    const int count = int(max(int64_t(0), min(total, start + chunk) - start));
    if (count == 0) {
        if (lane == 0) A.meta[2 * w] = make_int4(0, 0, 0, 0);
        return;
    }

    // each lane's cursor: the sequence of flattened block start + lane (+ 32, ...)
    int cb;
    int64_t cbase;  // blocks before sequence cb
    {
        int t = 0;
        for (int i = 0; i < kWarps; ++i)
            t += __popc(__ballot_sync(0xffffffffu, prefix[i * 32 + lane] <= start));
        cb = (t - 1) * per;  // threads without sequences share the last prefix: still its end
        cbase = prefix[t - 1];
    }
    Seq cs = load_seq(A, min(cb, A.B - 1), S::kRows);
    auto next_entry = [&](int64_t f) -> Entry {
        Entry e;
        while (cb < A.B && f >= cbase + cs.blocks(A.H)) {
            cbase += cs.blocks(A.H);
            ++cb;
            if (cb < A.B) cs = load_seq(A, cb, S::kRows);
        }
        e.b = cb;
        e.seg = 0;
        e.blk = 0;
        e.line = 0;
        e.sk = e.lg = 0.0f;
        if (cb >= A.B) return e;
        const uint64_t rem = uint64_t(f - cbase);
        e.seg = int(rem / uint32_t(cs.nb));
        e.blk = cs.lo + int(rem - uint64_t(e.seg) * uint32_t(cs.nb));
        if (e.blk * kPage < cs.len) {
            const int page = A.table[int64_t(cb) * A.max_pages + e.blk], head = e.seg / cs.tiles;
            if (page < 0 || page >= A.num_pages) {
                record(8);
                e.sk = e.lg = __int_as_float(0x7fffffff);
            } else {
                e.line = (page * A.H + head) * int(S::kTile / 128);
                e.sk = A.k_scale[int64_t(page) * A.H + head];
                e.lg = log2_scale(A.v_scale[int64_t(page) * A.H + head]);
            }
        }
        return e;
    };
    Entry cur = next_entry(start + lane), nxt = cur;

    // tile u of the worker (u = 2 * block + (0 K, 1 V)) goes to slot u % kSlots.  A tile is read
    // once, but by the few others of its head: first to leave L2 (535 MB 124 -> 119 us).
    const uint64_t once = l2_policy_evict_first();
    auto issue = [&](int u, int first) {
        const int i = (u >> 1) - first;
        const int line = __shfl_sync(0xffffffffu, i < 32 ? cur.line : nxt.line, i & 31);
        if ((u >> 1) < count && lane == 0) {
            const uint32_t bar = bars + 8 * uint32_t(u % kSlots);
            mbar_arrive_expect_tx(bar, S::kTile);
            tma_load_2d_hint(ring_addr + uint32_t(u % kSlots) * S::kTile, (u & 1) ? &tm_v : &tm_k, bar, 0, line, once);
        }
    };
    __syncwarp();
    for (int u = 0; u < kSlots; ++u) issue(u, 0);
    if (count > 32 - kSlots) nxt = next_entry(start + 32 + lane);

    // The reads of a tile are over before TMA writes its slot again: without the proxy fence a read
    // still in flight can be overtaken.
    auto release = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
    };

    bool ok = true;
    int window = 0, done = 0;         // first block of `cur`, tiles consumed
    int seg_b = -1, seg = -1;         // the open segment
    int seg_i = 0, seg_blk = 0;       // the block of the worker it was opened at, its index in the sequence
    bool split = false;               // this worker began a segment that goes on elsewhere
    Seq sq{};
    int head = 0, row0 = 0, tile_first = 0, tile_last = -1, all_first = 0, all_last = -1;
    uint32_t qf[NT][kSteps][2];
    float row_c[NT][2], m[NT][2], w_ref[NT][2], l[NT][2], acc[NT][kMT][4];
    int row_first[NT][2], row_last[NT][2];

    auto arrived = [&]() -> const uint8_t * {
        ok = mbar_wait(bars + 8 * uint32_t(done % kSlots), uint32_t(done / kSlots) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        return ring + (done % kSlots) * S::kTile;
    };

    auto open_segment = [&](int b, int sg) {
        if (b != seg_b) sq = load_seq(A, b, kRows);
        head = sg / sq.tiles;
        row0 = (sg - head * sq.tiles) * kRows;
        const int rows = sq.n * A.G, pos0 = sq.len - sq.n;
        auto first_of = [&](int i) { return A.window > 0 ? max(0, pos0 + i - A.window + 1) : 0; };
        auto last_of = [&](int i) { return A.causal || pos0 + i < 0 ? pos0 + i : sq.len - 1; };
        const int i_lo = row0 / A.G, i_hi = min(rows - 1, row0 + kRows - 1) / A.G;
        tile_first = first_of(i_lo);
        all_first = first_of(i_hi);
        all_last = last_of(i_lo);
        tile_last = last_of(i_hi);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // this lane reads 16 channels (or 32) of row g; it holds the statistics of rows 2c, 2c + 1
            const int rr = row0 + 8 * n + g, i = rr / A.G;
            const bool valid = rr < rows;
            const T *src = static_cast<const T *>(A.q) + (int64_t(sq.ts) + i) * A.q_stride +
                           int64_t(head * A.G + rr - i * A.G) * D;
            float x[kQuads][16], top = 0.0f;
#pragma unroll
            for (int j = 0; j < kQuads; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (valid) load4(src + 16 * (c + 4 * j) + 4 * k, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[j][4 * k + e] = f[e];
                        top = fmaxf(top, fabsf(f[e]));
                    }
                }
            float up = 1.0f, down = 1.0f;
            if (A.dtype == 0) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                row_power(top, up, down);
            }
#pragma unroll
            for (int j = 0; j < kQuads; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float *f = &x[j][4 * k];
                    qf[n][4 * j + k][0] = h2(__floats2half2_rn(f[0] * up, f[1] * up));
                    qf[n][4 * j + k][1] = h2(__floats2half2_rn(f[2] * up, f[3] * up));
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                row_c[n][e] = A.sm_scale * kLog2e * __shfl_sync(0xffffffffu, down, 4 * (2 * c + e));
                const int rs = row0 + 8 * n + 2 * c + e, is = rs / A.G;
                row_first[n][e] = first_of(is);
                row_last[n][e] = rs < rows ? last_of(is) : -1;
                m[n][e] = w_ref[n][e] = -INFINITY;
                l[n][e] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kMT; ++k) acc[n][k][0] = acc[n][k][1] = acc[n][k][2] = acc[n][k][3] = 0.0f;
        }
    };

    // Writes the open segment's piece.
    auto close_segment = [&]() {
        const bool begins = seg_blk == sq.lo;
        const int64_t seg_end = start + seg_i - (seg_blk - sq.lo) + sq.nb;
        const bool whole = begins && seg_end <= start + count;
        const int rows = sq.n * A.G - row0;
        const int slot = 2 * w + (seg_i == 0 ? 0 : 1);
        if (begins && !whole) {
            split = true;
            if (lane == 0) {
                A.meta[2 * w] = make_int4(int((seg_end - 1) / chunk) - w + 1, slot, 0, 0);
                A.meta[2 * w + 1] = make_int4(sq.ts, head, row0, min(kRows, rows));
            }
        }
        // the lane's channels: 16 (or 8) from ch on, of rows 2c and 2c + 1
        const int ch = D == 128 ? 16 * ((g & 1) * 4 + (g >> 1)) : 8 * g;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
#pragma unroll
                for (int o = 4; o < 32; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const int rt = 8 * n + 2 * c + e;
                if (rt >= rows) continue;
                float f, power;
                power_of(w_ref[n][e], m[n][e], kPBits, f, power);
                if (whole) f = sum == 0.0f ? 0.0f : f / sum;
                auto out = [&](int k, int i) { return acc[n][k][i] * f * power; };
                if (whole) {
                    const int rr = row0 + rt, i = rr / A.G, hq = head * A.G + rr - i * A.G;
                    const int64_t at = (int64_t(sq.ts) + i) * (A.H * A.G) + hq;
                    T *dst = static_cast<T *>(A.o) + at * D + ch;
                    if (A.lse && g == 0) A.lse[at] = sum == 0.0f ? -INFINITY : (m[n][e] + log2f(sum)) * kLn2;
#pragma unroll
                    for (int k = 0; k < kMT; k += 4)
                        *reinterpret_cast<uint4 *>(dst + 2 * k) =
                            make_uint4(pack_out(out(k, e), out(k, 2 + e), T()), pack_out(out(k + 1, e), out(k + 1, 2 + e), T()),
                                       pack_out(out(k + 2, e), out(k + 2, 2 + e), T()), pack_out(out(k + 3, e), out(k + 3, 2 + e), T()));
                } else {
                    float *part = A.part + int64_t(slot) * S::kPart;
                    if (g == 0) {
                        part[kRows * D + rt] = m[n][e];
                        part[kRows * (D + 1) + rt] = sum;
                    }
#pragma unroll
                    for (int k = 0; k < kMT; k += 2)
                        *reinterpret_cast<float4 *>(part + rt * D + ch + 2 * k) =
                            make_float4(out(k, e), out(k, 2 + e), out(k + 1, e), out(k + 1, 2 + e));
                }
            }
    };

    if (w == A.quit) ok = false;
    for (int i = 0; ok && i < count; ++i) {
        if (i - window == 32) {
            cur = nxt;
            window += 32;
            nxt = next_entry(start + window + 32 + lane);
        }
        const int at = i - window;
        const int b = __shfl_sync(0xffffffffu, cur.b, at), sg = __shfl_sync(0xffffffffu, cur.seg, at);
        const int blk = __shfl_sync(0xffffffffu, cur.blk, at);
        const float sk = __shfl_sync(0xffffffffu, cur.sk, at), lg = __shfl_sync(0xffffffffu, cur.lg, at);
        if (b != seg_b || sg != seg) {
            if (seg_b >= 0) close_segment();
            open_segment(b, sg);
            seg_b = b;
            seg = sg;
            seg_i = i;
            seg_blk = blk;
        }
        const int t0 = blk * kPage;
        const bool seen = t0 <= tile_last && t0 + kPage > tile_first;
        const bool full = t0 >= all_first && t0 + kPage - 1 <= all_last;

        // ---- S^T = k8 . q: 16 keys by 8 rows a product
        float s[NT][4][4];
        const uint8_t *tile = arrived();
        if (!ok) break;
        if (seen) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][mt][0] = s[n][mt][1] = s[n][mt][2] = s[n][mt][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < kQuads; ++j) {
                    uint4 v[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int key = 16 * mt + 8 * y + (D == 128 ? (g & 1) * 4 + (g >> 1) : g);
                        const int chunk16 = D == 128 ? c + 4 * j : (key & 1) * 4 + c;
                        const int ln = D == 128 ? key : key >> 1;
                        v[y] = *reinterpret_cast<const uint4 *>(tile + ln * 128 + ((chunk16 ^ (ln & 7)) << 4));
                    }
                    const uint32_t w0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, w1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x0 = w0[k] ^ 0x80808080u, x1 = w1[k] ^ 0x80808080u;
                        const uint32_t a[4] = {bytes_to_h2(x0, 0x4140u), bytes_to_h2(x1, 0x4140u), bytes_to_h2(x0, 0x4342u),
                                               bytes_to_h2(x1, 0x4342u)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(s[n][mt], a, qf[n][4 * j + k][0], qf[n][4 * j + k][1]);
                    }
                }
            }
        }
        release();
        issue(done + kSlots, window);
        ++done;

        // ---- P = 2^(x + bias); pf: as the second operand, 8 keys by 8 rows each
        uint32_t pf[NT][8];
        if (seen) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[n][mt][e] * (row_c[n][e & 1] * sk);
                        if (!full) {
                            const int t = t0 + 16 * mt + 8 * (e >> 1) + (D == 128 ? (g & 1) * 4 + (g >> 1) : g);
                            if (t < row_first[n][e & 1] || t > row_last[n][e & 1]) x = -INFINITY;
                        }
                        s[n][mt][e] = x;
                        top[e & 1] = fmaxf(top[e & 1], x);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
                if (__any_sync(0xffffffffu, top[0] > m[n][0] || top[1] > m[n][1] || top[0] + lg > w_ref[n][0] ||
                                                top[1] + lg > w_ref[n][1])) {
                    float factor[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // a NaN is passed over, and -inf less 0 is left where nothing was seen yet
                        const float m_new = fmaxf(m[n][e], ceilf(top[e])), w_new = fmaxf(w_ref[n][e], ceilf(top[e] + lg));
                        l[n][e] *= ex2_approx(m[n][e] - (m_new == -INFINITY ? 0.0f : m_new));
                        factor[e] = ex2_approx(w_ref[n][e] - (w_new == -INFINITY ? 0.0f : w_new));
                        m[n][e] = m_new;
                        w_ref[n][e] = w_new;
                    }
                    if (__any_sync(0xffffffffu, factor[0] != 1.0f || factor[1] != 1.0f)) {
#pragma unroll
                        for (int k = 0; k < kMT; ++k) {
                            acc[n][k][0] *= factor[0];
                            acc[n][k][1] *= factor[1];
                            acc[n][k][2] *= factor[0];
                            acc[n][k][3] *= factor[1];
                        }
                    }
                }
                // at: the exponent of P at x = m
                float bias[2], at[2], sum[2] = {0.0f, 0.0f};
                bool apart[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    bias[e] = kPBits - (w_ref[n][e] == -INFINITY ? 0.0f : w_ref[n][e]) + lg;
                    at[e] = bias[e] + (m[n][e] == -INFINITY ? 0.0f : m[n][e]);
                    apart[e] = !(at[e] >= kAtLeast);
                }
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float z[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = s[n][mt][2 * y + e];
                            z[e] = ex2_approx(x + bias[e]);
                            if (!full && x == -INFINITY) z[e] = 0.0f;  // whatever the block's scale
                            sum[e] += z[e];
                        }
                        pf[n][2 * mt + y] = transpose8x8(h2(__floats2half2_rn(z[0], z[1])));
                    }
                if (__any_sync(0xffffffffu, apart[0] || apart[1])) {  // P may vanish where p does not: such rows sum p
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (!apart[e]) continue;
                        at[e] = sum[e] = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = s[n][i >> 1][2 * (i & 1) + e];
                            sum[e] += ex2_approx(x - (m[n][e] == -INFINITY ? 0.0f : m[n][e]));
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) l[n][e] = fmaf(sum[e], ex2_approx(-at[e]), l[n][e]);
            }
        }

        // ---- acc^T += v8^T . P^T: 16 channels by 8 rows a product
        tile = arrived();
        if (!ok) break;
        if (seen) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // 16 keys
                uint32_t vw[4][D / 32];       // 4 keys x D / 8 channels of this lane
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int in8 = D == 128 ? c + 4 * (y & 1) : 2 * c + (y & 1);
                    const int key = 16 * kk + 8 * (y >> 1) + in8;
                    if (D == 128) {
                        const int chunk16 = (g & 1) * 4 + (g >> 1);
                        const uint4 v =
                            *reinterpret_cast<const uint4 *>(tile + key * 128 + ((chunk16 ^ (key & 7)) << 4));
                        vw[y][0] = v.x;
                        vw[y][1] = v.y;
                        vw[y][D / 32 - 2] = v.z;
                        vw[y][D / 32 - 1] = v.w;
                    } else {
                        const int ln = key >> 1, chunk16 = (key & 1) * 4 + (g >> 1);
                        const uint2 v = *reinterpret_cast<const uint2 *>(
                            tile + ln * 128 + ((chunk16 ^ (ln & 7)) << 4) + 8 * (g & 1));
                        vw[y][0] = v.x;
                        vw[y][1] = v.y;
                    }
                }
#pragma unroll
                for (int q4 = 0; q4 < D / 32; ++q4) {
                    uint32_t lo[2], hi[2];  // channels 4 q4 + {0, 1}, {2, 3} of both key pairs
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t w0 = vw[2 * y][q4], w1 = vw[2 * y + 1][q4];
                        lo[y] = __byte_perm(w0, w1, 0x5140) ^ 0x80808080u;
                        hi[y] = __byte_perm(w0, w1, 0x7362) ^ 0x80808080u;
                    }
                    const uint32_t a[4] = {bytes_to_h2(lo[0], 0x4140u), bytes_to_h2(lo[0], 0x4342u), bytes_to_h2(lo[1], 0x4140u),
                                           bytes_to_h2(lo[1], 0x4342u)};
                    const uint32_t b4[4] = {bytes_to_h2(hi[0], 0x4140u), bytes_to_h2(hi[0], 0x4342u), bytes_to_h2(hi[1], 0x4140u),
                                            bytes_to_h2(hi[1], 0x4342u)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(acc[n][2 * q4], a, pf[n][2 * kk], pf[n][2 * kk + 1]);
                        mma16816(acc[n][2 * q4 + 1], b4, pf[n][2 * kk], pf[n][2 * kk + 1]);
                    }
                }
            }
        }
        release();
        issue(done + kSlots, window);
        ++done;
    }
    if (ok) {
        close_segment();
    } else {
        if (lane == 0) record(6);
        // the tiles still in flight must land before the block's shared memory is given up
        for (int u = done; u < min(done + kSlots, 2 * count); ++u)
            drain_wait(bars + 8 * uint32_t(u % kSlots), uint32_t(u / kSlots) & 1u);
        // what others join with this warp's pieces is to be NaN, whichever of them it wrote
        __syncwarp();
        if (lane < kRows)
            for (int slot = 2 * w; slot < 2 * w + 2; ++slot)
                A.part[int64_t(slot) * S::kPart + kRows * D + lane] = __int_as_float(0x7fffffff);
    }
    if (!split && lane == 0) A.meta[2 * w] = make_int4(0, 0, 0, 0);
}

__device__ __forceinline__ void load_floats(const float *p, float (&v)[4])
{
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load_floats(const float *p, float (&v)[2])
{
    const float2 x = *reinterpret_cast<const float2 *>(p);
    v[0] = x.x; v[1] = x.y;
}

// Joins the pieces of the segments, of ROWS rows at most, that a worker began and others went on
// with: workers blockIdx.x, blockIdx.x + gridDim.x, ....  A piece is acc [ROWS][D], m [ROWS], l [ROWS].  The warps take the rows, and share a row's pieces
// where there are fewer rows.
constexpr int kCombineWarps = 8, kCombineThreads = 32 * kCombineWarps;
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kCombineThreads, 3) cache_combine_kernel(const CacheAttnArgs A, int workers)
{
    constexpr int kPart = ROWS * (D + 2), kPer = D / 32;
    __shared__ float sums[kCombineWarps][D];
    chain_begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // lane k looks at worker blockIdx.x + k * gridDim.x; both words come at once (the second may be old, unless used)
    int4 mine = make_int4(0, 0, 0, 0), place = mine;
    if (blockIdx.x + lane * gridDim.x < workers) {
        mine = A.meta[2 * (blockIdx.x + lane * gridDim.x)];
        place = A.meta[2 * (blockIdx.x + lane * gridDim.x) + 1];
    }
    uint32_t found = __ballot_sync(0xffffffffu, mine.x > 0);
    while (found) {
        const int k = __ffs(found) - 1, w = blockIdx.x + k * gridDim.x;
        found &= found - 1;
        const int pieces = __shfl_sync(0xffffffffu, mine.x, k), slot0 = __shfl_sync(0xffffffffu, mine.y, k);
        // first token, head, row of the segment in its head, its rows
        const int first = __shfl_sync(0xffffffffu, place.x, k), head = __shfl_sync(0xffffffffu, place.y, k);
        const int row0 = __shfl_sync(0xffffffffu, place.z, k), rows = __shfl_sync(0xffffffffu, place.w, k);
        int groups = 1;
        while (groups < rows && groups < kCombineWarps) groups *= 2;
        const int subs = kCombineWarps / groups, sub = warp / groups;
        for (int r = warp % groups; r < (subs > 1 ? groups : rows); r += groups) {
            auto part_of = [&](int p) { return A.part + int64_t(p == 0 ? slot0 : 2 * (w + p)) * kPart; };
            // A lane adds up kPer neighbouring channels of a row, kBatch pieces in flight at a time; the
            // first batch is on its way while the weights are found.
            constexpr int kBatch = 8;
            float v[kBatch][kPer], vm[kBatch], big = -INFINITY, total = 0.0f, out[kPer];
            auto load = [&](int p0) {
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int p = p0 + q * subs;
                    vm[q] = -INFINITY;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) v[q][e] = 0.0f;
                    if (p < pieces && r < rows) {
                        const float *part = part_of(p);
                        vm[q] = part[ROWS * D + r];
                        load_floats(part + r * D + lane * kPer, v[q]);
                    }
                }
            };
            load(sub);
#pragma unroll
            for (int e = 0; e < kPer; ++e) out[e] = 0.0f;
            float own = -INFINITY;  // the lane's maximum, which its total is relative to
            if (r < rows) {
                for (int p = lane; p < pieces; p += 32) {
                    const float *part = part_of(p);
                    const float pm = part[ROWS * D + r], pl = part[ROWS * (D + 1) + r];
                    const float next = fmaxf(own, pm), to = next == -INFINITY ? 0.0f : next;
                    total = total * ex2_approx(own - to) + pl * ex2_approx(pm - to);
                    own = next;
                }
                big = own;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            }
            const float ref = big == -INFINITY ? 0.0f : big;
            if (r < rows) {
                total *= ex2_approx(own - ref);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            }
            for (int p0 = sub;;) {
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const float f = ex2_approx(vm[q] - ref);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) out[e] = fmaf(f, v[q][e], out[e]);
                }
                p0 += kBatch * subs;
                if (p0 >= pieces) break;
                load(p0);
            }
            if (subs > 1) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) sums[warp][lane * kPer + e] = out[e];
                __syncthreads();
                if (sub == 0)
                    for (int y = 1; y < subs; ++y)
#pragma unroll
                        for (int e = 0; e < kPer; ++e) out[e] += sums[warp + y * groups][lane * kPer + e];
                __syncthreads();
            }
            if (r >= rows || sub > 0) continue;
            const float f = total == 0.0f ? 0.0f : 1.0f / total;
            const int rr = row0 + r, i = rr / A.G;
            const int64_t at = (int64_t(first) + i) * (A.H * A.G) + head * A.G + rr - i * A.G;
            uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(A.o) + at * D + lane * kPer);
#pragma unroll
            for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack_out(out[e] * f, out[e + 1] * f, T());
            if (A.lse && lane == 0) A.lse[at] = total == 0.0f ? -INFINITY : (big + log2f(total)) * kLn2;
        }
    }
}

// One wave of blocks looks after all workers: as a block for each worker, most of which have
// nothing to join, it took 14 us after 1776 workers.
template <typename T, int D, int ROWS>
cudaError_t launch_combine(const CacheAttnArgs &a, int workers, int sms, cudaStream_t st)
{
    return launch_chained(cache_combine_kernel<T, D, ROWS>, dim3(unsigned(std::min(workers, 6 * sms))),
                          kCombineThreads, 0, st, a, workers);
}

size_t meta_bytes(int sms) { return (size_t(sms) * kMaxWarps * 2 * sizeof(int4) + 255) & ~size_t(255); }

bool many_rows(int64_t T, int B, int G) { return B <= kCacheChunkMaxSeqs && T * G > int64_t(kFewRows) * B; }
bool two_tiles(int64_t T, int B, int G) { return T * G > int64_t(8) * B; }  // where most segments have over eight rows

template <int D>
size_t part_bytes(int sms, int64_t T, int B, int G)
{
    if (many_rows(T, B, G)) return cache_chunk_part_bytes(sms, D);
    const size_t each = two_tiles(T, B, G) ? size_t(Sizes<D, 2>::kWarps) * Sizes<D, 2>::kPart
                                           : size_t(Sizes<D, 1>::kWarps) * Sizes<D, 1>::kPart;
    return size_t(2) * sms * each * 4;
}

template <typename T, int D, int NT>
cudaError_t launch_for(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const CacheAttnArgs &a, int sms, cudaStream_t st)
{
    using S = Sizes<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(S::kAlloc));
    if (e != cudaSuccess) return e;
    e = launch_chained(cache_attn_kernel<T, D, NT>, dim3(unsigned(sms)), S::kThreads, S::kAlloc, st, tm_k, tm_v, a);
    if (e != cudaSuccess) return e;
    return launch_combine<T, D, S::kRows>(a, sms * S::kWarps, sms, st);
}

template <typename T, int D>
cudaError_t launch_any(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const CacheAttnArgs &a, int sms, cudaStream_t st)
{
    if (many_rows(a.T, a.B, a.G)) return launch_cache_chunk(a, sms, st);
    if (two_tiles(a.T, a.B, a.G)) return launch_for<T, D, 2>(tm_k, tm_v, a, sms, st);
    return launch_for<T, D, 1>(tm_k, tm_v, a, sms, st);
}

}  // namespace

size_t cache_attn_workspace(int sms, int64_t T, int B, int G, int d)
{
    return meta_bytes(sms) + (d == 128 ? part_bytes<128>(sms, T, B, G) : part_bytes<64>(sms, T, B, G));
}

cudaError_t launch_cache_attn(const CUtensorMap &tm_k, const CUtensorMap &tm_v, CacheAttnArgs a, void *workspace,
                              cudaStream_t st)
{
    const int sms = device_sms();
    if (sms < 1) return cudaErrorNoDevice;
    a.meta = static_cast<int4 *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + meta_bytes(sms));
    if (a.dtype == 0)
        return a.d == 128 ? launch_any<__nv_bfloat16, 128>(tm_k, tm_v, a, sms, st)
                          : launch_any<__nv_bfloat16, 64>(tm_k, tm_v, a, sms, st);
    return a.d == 128 ? launch_any<__half, 128>(tm_k, tm_v, a, sms, st) : launch_any<__half, 64>(tm_k, tm_v, a, sms, st);
}

cudaError_t read_and_clear_cache_attn_status(int *status)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(status, g_cache_attn_status, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_cache_attn_status, &zero, sizeof(int));
}

}  // namespace sa
