// sa_cache_chunk.cu -- attention of many query rows over the paged INT8 cache for sm_100a.
//
// The mathematics is that of sa_cache_attn.cu, on the 5th-generation tensor cores: S = q . k8 and
// acc += P . v8 are tcgen05 kind::f16 products of fp16 operands with fp32 accumulators in tensor
// memory.  A segment is 256 rows (two tiles of 128, A and B) of one sequence and key/value head,
// a row being a query token and one of the query heads that share the head, token-major; a step
// is 128 keys (two blocks).  Both tiles read one stream of K and V tiles.
//
// What bounds it: at d = 128 a step costs each SM 2048 cycles of tensor core, 2048 of ex2 (32768
// of them, 16 a cycle) and about 2050 of shared memory (Q and K for S, V for P . V, and the
// writing of the fp16 tiles), so all three have to run at once:
//   * warps 0-3 and 4-7: softmax of tile A and B, a thread owning a row (its 128 scores of a step
//     in registers): maximum, exponentials, P to tensor memory, rescaling of acc, epilogue;
//   * warps 8-11: the codes of a block, brought by TMA (warp 14, a ring of four 64-token tiles),
//     become fp16 tiles in shared memory (a ring of four, K and V in turn) in the 128-byte
//     swizzle that the tensor core reads: K as a K-major operand, V, whose channels are
//     contiguous, as an MN-major one;
//   * warp 12 issues S, warp 13 P . V.
// P is the A operand from tensor memory, which halves P . V's reading of shared memory.  S has
// one buffer for both tiles in turn, which staggers the two softmax groups by half a step.
//
// Rounding.  P is rounded to fp16 as 2^5 * p * scale_v / u, u a running reference of the value
// scales (a power of two, raised when a scale exceeds 4 u) and p relative to a reference m of the row's maximum
// (raised when the maximum exceeds m + 8, in powers of two), so it stays within 2^15 and acc is
// rescaled rarely; relative error 2^-11, subnormals below 2^-19 of the reference.  The factor is
// folded into the exponent, and a block's sum of p divided by it again in fp32.
//
// Work.  The steps of all segments, laid out one after another (sequence, head, rows), are cut
// into equal ranges, one for each SM, as in sa_cache_attn.cu; pieces of segments that two or more
// blocks share are joined by the combine kernel in a fixed order.  Every role walks the same
// pieces on its own.
#include <cstdint>

#include "sa_cache_attn.cuh"
#include "sa_internal.h"
#include "sa_ptx.cuh"

namespace sa {

__device__ int g_cache_chunk_status;  // 0 = OK, 6 = a bounded wait expired, 8 = bad index

namespace {

constexpr int kThreads = 512;
constexpr int kWarpConvert = 8, kWarpQK = 12, kWarpPV = 13, kWarpLoad = 14;
constexpr int kStages = 4;  // fp16 tiles
constexpr int kRaw = 4;     // 64-token tiles of codes
constexpr int kRowsSeg = 256;
constexpr uint32_t kTmemCols = 512, kColS = 0;
__host__ __device__ constexpr uint32_t col_p(int t) { return 128u + 64u * uint32_t(t); }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * uint32_t(t); }
constexpr uint32_t kRegsSoftmax = 208, kRegsConvert = 56, kRegsIssue = 40, kLaunchRegs = 128;
static_assert(128 * (2 * kRegsSoftmax + kRegsConvert + kRegsIssue) <= kLaunchRegs * kThreads,
              "the register split must fit the registers the block is launched with");
constexpr float kGrow = 8.0f;

constexpr int kBarQFull = 0, kBarKvFull = 2, kBarKvEmpty = kBarKvFull + kStages, kBarSFull = kBarKvEmpty + kStages,
              kBarSEmpty = kBarSFull + 2, kBarPFull = kBarSEmpty + 1, kBarPvDone = kBarPFull + 2,
              kBarOFull = kBarPvDone + 2, kBarOEmpty = kBarOFull + 2, kBarRawFull = kBarOEmpty + 2,
              kBarRawEmpty = kBarRawFull + kRaw, kNumBars = kBarRawEmpty + kRaw;

template <int D>
struct Sizes {
    static constexpr int kSub = D / 64;                      // 64-channel halves of a tile
    static constexpr uint32_t kSubBytes = 128 * 128;         // 128 rows x 128 bytes
    static constexpr uint32_t kTileBytes = kSub * kSubBytes; // a Q, K or V tile in fp16
    static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kTileBytes;
    static constexpr uint32_t kRawBytes = 64 * D;
    static constexpr uint32_t kOffRaw = kOffKv + kStages * kTileBytes;
    static constexpr uint32_t kOffBar = kOffRaw + kRaw * kRawBytes;
    static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr uint32_t kAlloc = kOffMisc + 16 + 1024;
    static constexpr int kPart = kRowsSeg * (D + 2);
};
static_assert(Sizes<128>::kAlloc <= 227 * 1024 - 1200, "shared memory per CTA");
static_assert(4 * kCacheChunkMaxSeqs <= kStages * Sizes<64>::kTileBytes, "the costs fit the ring before it is used");

template <uint32_t NR>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(NR)); }
template <uint32_t NR>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(NR)); }

__device__ __forceinline__ void record(int what) { atomicMax(&g_cache_chunk_status, what); }

struct Seq {
    int ts, n, len, pairs;
};
__device__ __forceinline__ Seq load_seq(const CacheAttnArgs &A, int b)
{
    Seq s;
    if (!load_span(A, b, s.ts, s.n, s.len)) record(8);
    s.pairs = (s.n * A.G + kRowsSeg - 1) / kRowsSeg;
    return s;
}

// What segment p of a sequence sees: blocks [blo, bhi), at least one step.
struct Reach {
    int blo, bhi;
    __device__ int steps() const { return max(1, (bhi - blo + 1) / 2); }
};
__device__ __forceinline__ Reach reach_of(const CacheAttnArgs &A, const Seq &s, int p)
{
    const int rows = s.n * A.G, pos0 = s.len - s.n;
    const int i_lo = p * kRowsSeg / A.G, i_hi = min(rows - 1, p * kRowsSeg + kRowsSeg - 1) / A.G;
    const int last = A.causal ? pos0 + i_hi : s.len - 1;
    const int first = A.window > 0 ? max(0, pos0 + i_lo - A.window + 1) : 0;
    Reach r;
    r.blo = first / kPage;
    r.bhi = last < first ? r.blo : last / kPage + 1;
    return r;
}

// The pieces of this block's range, one after another.  Each warp has its own in shared memory,
// stepped by lane 0: the softmax warps have no registers to spare for it.
struct Walk {
    int b, h, p, off;   // segment (sequence, head, rows) and the step it goes on with
    int64_t pos, end;   // flattened steps
    Seq s;
    Reach r;
    int count;          // steps of the piece
    bool begins, ends;
    int pieces;         // pieces before this one

    __device__ bool open(const CacheAttnArgs &A)
    {
        __syncwarp();
        if (pos >= end) return false;
        if ((threadIdx.x & 31) == 0) prepare(A);
        __syncwarp();
        return true;
    }
    __device__ void next(const CacheAttnArgs &A)
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) step(A);
    }
    __device__ int tiles(const CacheAttnArgs &A) const { return s.n * A.G - p * kRowsSeg > 128 ? 2 : 1; }

private:
    __device__ void prepare(const CacheAttnArgs &A)
    {
        r = reach_of(A, s, p);
        const int st = r.steps();
        count = int(min(int64_t(st - off), end - pos));
        begins = off == 0;
        ends = off + count == st;
    }
    __device__ void step(const CacheAttnArgs &A)
    {
        pos += count;
        off = 0;
        ++pieces;
        if (pos >= end) return;  // whatever follows is another block's
        if (++p < s.pairs) return;
        p = 0;
        if (++h < A.H) return;
        h = 0;
        do s = load_seq(A, ++b);
        while (s.n == 0 && b + 1 < A.B);
    }
};

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Orders later uses of r after a tcgen05.wait::ld (the array passes through the statement).
__device__ __forceinline__ void regs_ready(uint32_t (&r)[32])
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ float fl_of(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ float max64(const uint32_t (&a)[32], const uint32_t (&b)[32])
{
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(fl_of(a[k]), fl_of(b[k]));
#pragma unroll
    for (int i = 4; i < 32; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmax3(m[k], fl_of(a[i + k]), fl_of(b[i + k]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// fp16 pair, `a` in the low half
__device__ __forceinline__ uint32_t pack_h2(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// 32 scores -> 16 words of P; returns the sum of 2^(s * c + bias).
__device__ __forceinline__ float p32(const uint32_t (&s)[32], float c, float bias, uint32_t *pw)
{
    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float y0, y1;
        fma2(y0, y1, fl_of(s[i]), fl_of(s[i + 1]), c, c, bias, bias);
        const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
        fma2(sum0, sum1, e0, e1, 1.0f, 1.0f, sum0, sum1);
        pw[i / 2] = pack_h2(e0, e1);
    }
    return sum0 + sum1;
}
// The same for any mask (bit i: key i seen) and scales: p apart from its factor f, unseen keys 0.
__device__ __forceinline__ float p32_any(const uint32_t (&s)[32], float c, float bias, float f, uint32_t keep, uint32_t *pw)
{
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float e0 = (keep >> i) & 1u ? ex2_approx(fmaf(fl_of(s[i]), c, bias)) : 0.0f;
        const float e1 = (keep >> (i + 1)) & 1u ? ex2_approx(fmaf(fl_of(s[i + 1]), c, bias)) : 0.0f;
        sum += e0 + e1;
        pw[i / 2] = pack_h2((keep >> i) & 1u ? e0 * f : 0.0f, (keep >> (i + 1)) & 1u ? e1 * f : 0.0f);
    }
    return sum;
}

// bits lo..hi-1 (clamped) of a 32-bit mask whose bit 0 is key `at`
__device__ __forceinline__ uint32_t keep_bits(int at, int lo, int hi)
{
    const int a = max(0, lo - at), b = min(32, hi - at);
    if (a >= b) return 0u;
    return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const CacheAttnArgs A)
{
    using S = Sizes<D>;
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128, false), kIdescPV = idesc_f16_f32(128, D, true);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int64_t range[2];     // flattened start, total
    __shared__ int first[4];         // sequence, head, segment and step of the start
    __shared__ Walk walks[kThreads / 32];
    int *cost = reinterpret_cast<int *>(smem + S::kOffKv);  // steps of a sequence's segments, of one head
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + S::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    auto bar = [&](int i) -> uint32_t { return sbase + S::kOffBar + 8u * uint32_t(i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar(kBarKvFull + i), 4);
            mbar_init(bar(kBarKvEmpty + i), 1);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(bar(kBarRawFull + i), 1);
            mbar_init(bar(kBarRawEmpty + i), 4);
        }
        mbar_init(bar(kBarSEmpty), 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(kBarQFull + t), 4);
            mbar_init(bar(kBarSFull + t), 1);
            mbar_init(bar(kBarPFull + t), 4);
            mbar_init(bar(kBarPvDone + t), 1);
            mbar_init(bar(kBarOFull + t), 1);
            mbar_init(bar(kBarOEmpty + t), 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpQK) tmem_alloc(sbase + S::kOffMisc, kTmemCols);
    // ---- the work: a warp sums a sequence's segments, or with many sequences each thread one's
    if (A.B > 64) {
        for (int b = threadIdx.x; b < A.B; b += kThreads) {
            const Seq s = load_seq(A, b);
            int sum = 0;
            for (int p = 0; p < s.pairs; ++p) sum += reach_of(A, s, p).steps();
            cost[b] = sum;
        }
    } else for (int b = warp; b < A.B; b += kThreads / 32) {
        const Seq s = load_seq(A, b);
        int sum = 0;
        for (int p = lane; p < s.pairs; p += 32) sum += reach_of(A, s, p).steps();
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) cost[b] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        int64_t total = 0;
        for (int b = lane; b < A.B; b += 32) total += cost[b];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= A.H;
        const int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
        const int64_t start = min(total, chunk * blockIdx.x);
        if (lane == 0) {
            range[0] = start;
            range[1] = total;
        }
        if (start < total) {
            int64_t before = 0;
            int b = 0;
            for (; b < A.B; b += 32) {  // 32 sequences at a time: those that end at or before the start
                const int64_t mine = b + lane < A.B ? int64_t(cost[b + lane]) * A.H : 0;
                int64_t incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, before + incl <= start);
                const int n = past == 0xffffffffu ? 32 : __ffs(~past) - 1;
                if (n < 32) {
                    before += __shfl_sync(0xffffffffu, incl - mine, n);
                    b += n;
                    break;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            const Seq s = load_seq(A, b);
            int rem = int((start - before) % cost[b]);
            const int h = int((start - before) / cost[b]);
            int p = 0;
            for (; p < s.pairs; p += 32) {
                const int mine = p + lane < s.pairs ? reach_of(A, s, p + lane).steps() : 0;
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, incl <= rem);
                const int n = past == 0xffffffffu ? 32 : __ffs(~past) - 1;
                if (n < 32) {
                    rem -= __shfl_sync(0xffffffffu, incl - mine, n);
                    p += n;
                    break;
                }
                rem -= __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) {
                first[0] = b;
                first[1] = h;
                first[2] = p;
                first[3] = rem;
            }
        }
    }
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    const int64_t total = range[1], chunk = (total + gridDim.x - 1) / gridDim.x;
    Walk &w = walks[warp];
    if (lane == 0) {
        w.pos = range[0];
        w.end = min(total, chunk * (int64_t(blockIdx.x) + 1));
        w.pieces = 0;
        if (w.pos < w.end) {
            w.b = first[0];
            w.h = first[1];
            w.p = first[2];
            w.off = first[3];
            w.s = load_seq(A, w.b);
        }
    }
    bool ok = true;  // the same in all lanes of a warp
    auto wait = [&](int i, uint32_t parity) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, abort_flag));
        return ok;
    };

    if (warp >= kWarpQK) {
        regs_dec<kRegsIssue>();
        if (warp == kWarpQK) {
            // ------------------------------------------------------------ S_A(j), S_B(j), S_A(j + 1), ...
            uint32_t g = 0, u = 0, q[2] = {0, 0};
            for (; ok && w.open(A); w.next(A)) {
                const int nt = w.tiles(A);
                for (int t = 0; t < nt && ok; ++t) wait(kBarQFull + t, q[t]++);
                for (int j = 0; j < w.count && ok; ++j, ++g) {
                    const uint32_t st = (2 * g) % kStages;
                    wait(kBarKvFull + st, ((2 * g) / kStages));
                    const uint32_t kb = sbase + S::kOffKv + st * S::kTileBytes;
                    for (int t = 0; t < nt && ok; ++t, ++u) {
                        if (u >= 1) wait(kBarSEmpty, (u - 1));
                        if (!ok) break;
                        tc_fence_after();
                        if (lane != 0) continue;
                        const uint32_t qa = sbase + S::kOffQ + uint32_t(t) * S::kTileBytes;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t at = uint32_t(kk / 4) * S::kSubBytes + uint32_t(kk % 4) * 32;
                            mma_f16(tmem + kColS, sdesc(qa + at, 1024, SWZ_128B), sdesc(kb + at, 1024, SWZ_128B),
                                    kIdescQK, kk > 0);
                        }
                        tc_commit(bar(kBarSFull + t));
                    }
                    if (ok && lane == 0) tc_commit(bar(kBarKvEmpty + st));
                }
            }
        } else if (warp == kWarpPV) {
            // ------------------------------------------------------------ acc += P . V
            uint32_t g = 0, c[2] = {0, 0}, o[2] = {0, 0};
            for (; ok && w.open(A); w.next(A)) {
                const int nt = w.tiles(A);
                for (int j = 0; j < w.count && ok; ++j, ++g) {
                    const uint32_t st = (2 * g + 1) % kStages;
                    wait(kBarKvFull + st, ((2 * g + 1) / kStages));
                    const uint32_t vb = sbase + S::kOffKv + st * S::kTileBytes;
                    for (int t = 0; t < nt && ok; ++t) {
                        wait(kBarPFull + t, c[t]);
                        if (ok && j == 0 && o[t] >= 1) wait(kBarOEmpty + t, (o[t] - 1));
                        if (!ok) break;
                        ++c[t];
                        if (lane != 0) continue;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_f16_ta(tmem + col_o(t), tmem + col_p(t) + 8 * kk,
                                       sdesc_mn16(vb + 2048 * kk, S::kSubBytes, 1024), kIdescPV,
                                       (j > 0 || kk > 0) ? 1u : 0u);
                        tc_commit(bar(kBarPvDone + t));
                    }
                    if (ok && lane == 0) tc_commit(bar(kBarKvEmpty + st));
                }
                for (int t = 0; t < nt && ok; ++t) {
                    if (lane == 0) tc_commit(bar(kBarOFull + t));
                    ++o[t];
                }
            }
        } else if (warp == kWarpLoad) {
            // ------------------------------------------------------------ codes of K0, K1, V0, V1 of each step
            uint32_t u = 0;
            for (; ok && w.open(A); w.next(A)) {
                int line_l = 0;  // lane i: block i of a window of 32, its first 128-byte line
                for (int j = 0; j < w.count && ok; ++j) {
                    if (j % 16 == 0) {
                        const int blk = w.r.blo + 2 * (w.off + j) + lane;
                        line_l = 0;
                        if (blk < w.r.bhi && 2 * j + lane < 2 * w.count) {
                            const int page = A.table[int64_t(w.b) * A.max_pages + blk];
                            if (page < 0 || page >= A.num_pages)
                                record(8);
                            else
                                line_l = (page * A.H + w.h) * (D / 2);
                        }
                    }
#pragma unroll 1
                    for (int k = 0; k < 4 && ok; ++k, ++u) {
                        const int line = __shfl_sync(0xffffffffu, line_l, 2 * (j % 16) + (k & 1));
                        const uint32_t st = u % kRaw;
                        if (u >= kRaw) wait(kBarRawEmpty + st, ((u / kRaw) - 1));
                        if (ok && lane == 0) {
                            mbar_arrive_expect_tx(bar(kBarRawFull + st), S::kRawBytes);
                            tma_load_2d(sbase + S::kOffRaw + st * S::kRawBytes, k < 2 ? &tm_k : &tm_v,
                                        bar(kBarRawFull + st), 0, line);
                        }
                    }
                }
            }
            // tiles in flight land before the block's shared memory is given up
            if (!ok)
                for (uint32_t v = u > kRaw ? u - kRaw : 0; v < u; ++v)
                    for (int i = 0; i < 1 << 20 && !mbar_try_wait(bar(kBarRawFull + v % kRaw), (v / kRaw) & 1); ++i) {
                    }
        }
    } else if (warp >= kWarpConvert) {
        // ---------------------------------------------------------------- codes to fp16 tiles
        regs_dec<kRegsConvert>();
        constexpr int kRowChunks = D / 16;           // 16-byte chunks of a row of codes
        constexpr int kRowsPass = 128 / kRowChunks;  // rows that the 128 threads take at once
        constexpr int kPasses = 64 / kRowsPass;
        const int tid = threadIdx.x - 32 * kWarpConvert, row = tid / kRowChunks, chunk16 = tid % kRowChunks;
        // TMA's swizzle of 128-byte lines (a line is a row, or two rows at d = 64); a pass is 16 lines
        const int line = tid / 8;
        const uint32_t from = uint32_t(line) * 128 + ((uint32_t(tid % 8) ^ uint32_t(line & 7)) << 4);
        // the 16 values are two 16-byte chunks of a row; half of the threads write theirs in the
        // other order, so that a store instruction touches all banks once
        const uint32_t base = uint32_t(chunk16 / 4) * S::kSubBytes + uint32_t(row) * 128;
        const uint32_t c0 = uint32_t(chunk16 % 4) * 2;
        const bool swap = D == 128 ? chunk16 >= 4 : (row & 1) != 0;
        const uint32_t to0 = base + (((c0 + (swap ? 1 : 0)) ^ uint32_t(row & 7)) << 4);
        const uint32_t to1 = base + (((c0 + (swap ? 0 : 1)) ^ uint32_t(row & 7)) << 4);
        uint32_t u = 0, raw = 0;  // fp16 tiles written, tiles of codes read
        for (; ok && w.open(A); w.next(A)) {
            for (int j = 0; j < 2 * w.count && ok; ++j, ++u) {  // K and V of each step
                const uint32_t st = u % kStages;
                if (u >= kStages) wait(kBarKvEmpty + st, ((u / kStages) - 1));
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf, ++raw) {
                    const uint32_t rs = raw % kRaw;
                    if (ok) wait(kBarRawFull + rs, (raw / kRaw));
                    if (!ok) break;
                    const uint8_t *src = smem + S::kOffRaw + rs * S::kRawBytes + from;
                    uint8_t *tile = smem + S::kOffKv + st * S::kTileBytes + hf * 64 * 128;
                    uint4 v[kPasses];
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) v[i] = *reinterpret_cast<const uint4 *>(src + i * 16 * 128);
                    if (w.r.blo + 2 * (w.off + j / 2) + hf >= w.r.bhi) {  // no such block: codes 0
#pragma unroll
                        for (int i = 0; i < kPasses; ++i) v[i] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const uint32_t wd[4] = {v[i].x ^ 0x80808080u, v[i].y ^ 0x80808080u, v[i].z ^ 0x80808080u,
                                                v[i].w ^ 0x80808080u};
                        uint4 a, b;
                        a.x = bytes_to_h2(wd[0], 0x4140u);
                        a.y = bytes_to_h2(wd[0], 0x4342u);
                        a.z = bytes_to_h2(wd[1], 0x4140u);
                        a.w = bytes_to_h2(wd[1], 0x4342u);
                        b.x = bytes_to_h2(wd[2], 0x4140u);
                        b.y = bytes_to_h2(wd[2], 0x4342u);
                        b.z = bytes_to_h2(wd[3], 0x4140u);
                        b.w = bytes_to_h2(wd[3], 0x4342u);
                        *reinterpret_cast<uint4 *>(tile + to0 + i * kRowsPass * 128) = swap ? b : a;
                        *reinterpret_cast<uint4 *>(tile + to1 + i * kRowsPass * 128) = swap ? a : b;
                    }
                    // orders the writes before the tensor core's reads, and the reads of the codes
                    // before TMA's next writes: without it a read still in flight can be overtaken
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarRawEmpty + rs));
                }
                if (ok && lane == 0) mbar_arrive(bar(kBarKvFull + st));
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax of tile t
        regs_inc<kRegsSoftmax>();
        const int t = warp >> 2, wq = warp & 3;
        const int row = wq * 32 + lane;
        const uint32_t lane_addr = uint32_t(wq * 32) << 16;
        const uint32_t sa = tmem + lane_addr + kColS, pa = tmem + lane_addr + col_p(t), oa = tmem + lane_addr + col_o(t);
        uint8_t *qrow = smem + S::kOffQ + uint32_t(t) * S::kTileBytes + row * 128;
        uint32_t c = 0, o = 0;  // steps and pieces of this tile
        bool split = false;
        const int wk = int(blockIdx.x);
        for (; w.open(A); w.next(A)) {
            if (t >= w.tiles(A)) continue;
            int lo, hi;  // the keys that this row sees, [lo, hi); rows past the last see all, and are not written
            {
                const int rr = w.p * kRowsSeg + t * 128 + row, pos = w.s.len - w.s.n + rr / A.G;
                const bool valid = rr < w.s.n * A.G;
                hi = min(valid && A.causal ? pos + 1 : w.s.len, w.r.bhi * kPage);
                lo = valid && A.window > 0 ? max(0, pos - A.window + 1) : 0;
            }
            // ---- this row of q, fp16 (the tile is free: S of the last step before was read)
            float rc;
            {
                const int rr = w.p * kRowsSeg + t * 128 + row, i = rr / A.G;
                const bool valid = rr < w.s.n * A.G;
                const T *src = static_cast<const T *>(A.q) + (int64_t(w.s.ts) + i) * A.q_stride +
                               int64_t(w.h * A.G + rr - i * A.G) * D;
                float up = 1.0f, down = 1.0f, top = 0.0f;
                if (valid && A.dtype == 0) {
#pragma unroll 4
                    for (int k = 0; k < D; k += 4) {
                        float f[4];
                        load4(src + k, f);
                        top = fmax3(fmaxf(top, fabsf(f[0])), fabsf(f[1]), fmaxf(fabsf(f[2]), fabsf(f[3])));
                    }
                    row_power(top, up, down);
                }
                rc = A.sm_scale * kLog2e * down;
#pragma unroll 4
                for (int k = 0; k < D; k += 8) {
                    float f[8] = {};
                    if (valid) {
                        load4(src + k, *reinterpret_cast<float(*)[4]>(&f[0]));
                        load4(src + k + 4, *reinterpret_cast<float(*)[4]>(&f[4]));
                    }
                    uint4 v;
                    v.x = pack_h2(f[0] * up, f[1] * up);
                    v.y = pack_h2(f[2] * up, f[3] * up);
                    v.z = pack_h2(f[4] * up, f[5] * up);
                    v.w = pack_h2(f[6] * up, f[7] * up);
                    *reinterpret_cast<uint4 *>(qrow + (k / 64) * S::kSubBytes + ((((k / 8) & 7) ^ (row & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarQFull + t));
            }
            float m = -INFINITY, l = 0.0f, u = 0.0f;
            // Scales of 16 steps at a time, lane i those of block i: scale_k; f = 2^5 scale_v / u, its
            // logarithm and inverse.
            float sk_l = 0.0f, f_l = 0.0f, g_l = 0.0f, inv_l = 0.0f;
            for (int j = 0; j < w.count; ++j, ++c) {
                float su = 1.0f;
                if (j % 16 == 0) {
                    const int blk = w.r.blo + 2 * (w.off + j) + lane;
                    float sv = 0.0f;
                    sk_l = 0.0f;
                    if (blk < w.r.bhi && 2 * j + lane < 2 * w.count) {
                        const int page = A.table[int64_t(w.b) * A.max_pages + blk];
                        if (page < 0 || page >= A.num_pages) {
                            sk_l = sv = __int_as_float(0x7fffffff);
                        } else {
                            sk_l = A.k_scale[int64_t(page) * A.H + w.h];
                            sv = A.v_scale[int64_t(page) * A.H + w.h];
                        }
                    }
                    // the reference of the value scales; one that is not finite leaves it
                    const float top = __uint_as_float(
                        __reduce_max_sync(0xffffffffu, sv > 0.0f && sv < INFINITY ? __float_as_uint(sv) : 0u));
                    if (top > 4.0f * u) {
                        const float u_new = scale_ref(top);
                        su = u / u_new;
                        u = u_new;
                    }
                    f_l = sv == 0.0f ? 0.0f : 32.0f * (sv / u);
                    const bool plain = f_l > 1e-15f && f_l < INFINITY;
                    g_l = plain ? log2f(f_l) : 0.0f;
                    inv_l = plain ? 1.0f / f_l : 0.0f;  // 0: f must be applied apart from the exponent
                }
                const int jj = 2 * (j % 16), t0 = (w.r.blo + 2 * (w.off + j)) * kPage;
                const float c0 = rc * __shfl_sync(0xffffffffu, sk_l, jj), c1 = rc * __shfl_sync(0xffffffffu, sk_l, jj + 1);
                const float inv0 = __shfl_sync(0xffffffffu, inv_l, jj), inv1 = __shfl_sync(0xffffffffu, inv_l, jj + 1);
                const bool plain = inv0 > 0.0f && inv1 > 0.0f && lo <= t0 && hi >= t0 + 2 * kPage;

                if (ok) wait(kBarSFull + t, c);
                uint32_t s[4][32];
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32_nowait(sa + 32 * k, s[k]);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int k = 0; k < 4; ++k) regs_ready(s[k]);
                }
                const bool fast = __all_sync(0xffffffffu, plain);
                uint32_t keep[4];
                if (!fast) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        keep[k] = keep_bits(t0 + 32 * k, lo, hi);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((keep[k] >> e) & 1u)) s[k][e] = 0xff800000u;  // -inf
                    }
                }
                // the scales are not negative, so they commute with the maximum (0 * -inf is
                // a NaN, which fmaxf passes over)
                const float top = fmaxf(max64(s[0], s[1]) * c0, max64(s[2], s[3]) * c1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarSEmpty));

                float alpha = 1.0f;
                if (top > m + kGrow || (m == -INFINITY && top > m)) {
                    alpha = ex2_approx(m - top);
                    m = top;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                l *= alpha;
                // P's columns and acc are free once P . V of the step before is done
                if (c >= 1 && ok) wait(kBarPvDone + t, (c - 1));
                tc_fence_after();
                if (fast) {
                    const float g0 = __shfl_sync(0xffffffffu, g_l, jj) - ref, g1 = __shfl_sync(0xffffffffu, g_l, jj + 1) - ref;
                    uint32_t pw[32];
                    float s0 = p32(s[0], c0, g0, pw);
                    s0 += p32(s[1], c0, g0, pw + 16);
                    if (ok) tmem_st32(pa, pw);
                    float s1 = p32(s[2], c1, g1, pw);
                    s1 += p32(s[3], c1, g1, pw + 16);
                    if (ok) tmem_st32(pa + 32, pw);
                    l += s0 * inv0 + s1 * inv1;
                } else {
                    const float f0 = __shfl_sync(0xffffffffu, f_l, jj), f1 = __shfl_sync(0xffffffffu, f_l, jj + 1);
                    uint32_t pw[32];
                    l += p32_any(s[0], c0, -ref, f0, keep[0], pw) + p32_any(s[1], c0, -ref, f0, keep[1], pw + 16);
                    if (ok) tmem_st32(pa, pw);
                    l += p32_any(s[2], c1, -ref, f1, keep[2], pw) + p32_any(s[3], c1, -ref, f1, keep[3], pw + 16);
                    if (ok) tmem_st32(pa + 32, pw);
                }
                if (ok) {
                    const float f = alpha * su;
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            uint32_t r[32];
                            tmem_ld32_wait(oa + 32 * k, r);
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float x, y;
                                mul2(x, y, fl_of(r[e]), fl_of(r[e + 1]), f, f);
                                r[e] = __float_as_uint(x);
                                r[e + 1] = __float_as_uint(y);
                            }
                            tmem_st32(oa + 32 * k, r);
                        }
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarPFull + t));
            }
            // ---- epilogue of the piece
            if (ok) wait(kBarOFull + t, o);
            if (ok) {
                tc_fence_after();
                const int rr = w.p * kRowsSeg + t * 128 + row, i = rr / A.G;
                const bool valid = rr < w.s.n * A.G;
                const int64_t at = (int64_t(w.s.ts) + i) * (A.H * A.G) + w.h * A.G + rr - i * A.G;
                const bool whole = w.begins && w.ends;
                const int slot = 2 * wk + (w.pieces == 0 ? 0 : 1);
                const float f = whole ? (l == 0.0f ? 0.0f : u / (32.0f * l)) : u * 0.03125f;
                float *part = A.part + int64_t(slot) * S::kPart;
                if (w.begins && !w.ends) {
                    split = true;
                    if (t == 0 && wq == 0 && lane == 0)
                        A.meta[wk] = make_int4(w.b, w.h * w.s.pairs + w.p, int((w.pos + w.r.steps() - 1) / chunk), slot);
                }
                if (valid && whole && A.lse) A.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                if (valid && !whole) {
                    part[kRowsSeg * D + t * 128 + row] = m;
                    part[kRowsSeg * (D + 1) + t * 128 + row] = l;
                }
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t r[32];
                    tmem_ld32_wait(oa + 32 * k, r);
                    if (!valid) continue;
                    if (whole) {
                        T *dst = static_cast<T *>(A.o) + at * D + 32 * k;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(dst + e) =
                                make_uint4(pack_out(fl_of(r[e]) * f, fl_of(r[e + 1]) * f, T()),
                                           pack_out(fl_of(r[e + 2]) * f, fl_of(r[e + 3]) * f, T()),
                                           pack_out(fl_of(r[e + 4]) * f, fl_of(r[e + 5]) * f, T()),
                                           pack_out(fl_of(r[e + 6]) * f, fl_of(r[e + 7]) * f, T()));
                    } else {
                        float *dst = part + int64_t(t * 128 + row) * D + 32 * k;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + e) = make_float4(fl_of(r[e]) * f, fl_of(r[e + 1]) * f,
                                                                               fl_of(r[e + 2]) * f, fl_of(r[e + 3]) * f);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarOEmpty + t));
            ++o;
        }
        // tile A takes part in every piece, so it knows whether a segment was begun and not ended
        if (warp == 0 && lane == 0 && !split) A.meta[wk] = make_int4(0, 0, 0, 0);
    }
    if (lane == 0 && !ok) {
        *abort_flag = 1;
        record(6);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpQK) tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int D>
cudaError_t launch_for(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const CacheAttnArgs &a, int sms, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(cache_chunk_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(Sizes<D>::kAlloc));
    if (e != cudaSuccess) return e;
    cache_chunk_kernel<T, D><<<sms, kThreads, Sizes<D>::kAlloc, st>>>(tm_k, tm_v, a);
    return cudaGetLastError();
}

}  // namespace

size_t cache_chunk_part_bytes(int sms, int d)
{
    return size_t(2) * sms * size_t(d == 128 ? Sizes<128>::kPart : Sizes<64>::kPart) * 4;
}

cudaError_t launch_cache_chunk(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const CacheAttnArgs &a, int sms,
                               cudaStream_t st)
{
    if (a.dtype == 0)
        return a.d == 128 ? launch_for<__nv_bfloat16, 128>(tm_k, tm_v, a, sms, st)
                          : launch_for<__nv_bfloat16, 64>(tm_k, tm_v, a, sms, st);
    return a.d == 128 ? launch_for<__half, 128>(tm_k, tm_v, a, sms, st) : launch_for<__half, 64>(tm_k, tm_v, a, sms, st);
}

cudaError_t read_and_clear_cache_chunk_status(int *status)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(status, g_cache_chunk_status, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_cache_chunk_status, &zero, sizeof(int));
}

}  // namespace sa
