// sa_cache_chunk.cu -- attention of many query rows over the paged INT8 cache for sm_100a.
//
// The mathematics is that of sa_cache_attn.cu, on the 5th-generation tensor cores: S = q . k8 and
// acc += P . v8 are tcgen05 kind::f16 products of fp16 operands with fp32 accumulators in tensor
// memory.  A segment is 256 rows (two tiles of 128, A and B) of one sequence and key/value head,
// a row being a query token and one of the query heads that share the head, token-major; a step
// is 128 keys (two blocks).  Both tiles read one stream of K and V tiles.
//
// What bounds it: at d = 128 a step costs each SM 2048 cycles of tensor core, 2048 of ex2 (32768
// of them, 16 a cycle) and 2560 of shared memory (1024 for Q and K of S, 512 for V of P . V, 512 to
// write the fp16 tiles, 512 for the codes in and out), so all three have to run at once.  Measured,
// 1560 queries of 40 heads over 32760 tokens: 1004 us in a burst at 1965 MHz (1042 TFLOP/s, 3370 cycles
// a step), 1177 us at the power limit (1570 MHz, 889 TFLOP/s).  No unit is full (tensor core 56 % of the
// cycles, ex2 58 %): what sets the pace is the chain S - softmax - P . V with shared memory under it.
// Taken out to see: the exponentials 5 % less, half the tile writes 8 %, the copies of codes 14 %.  Who
// does what:
//   * warps 0-3 and 4-7: softmax of tile A and B, a thread owning a row (its 128 scores of a step
//     in registers): maximum, exponentials, P to tensor memory, rescaling of acc, epilogue;
//   * warps 8-11: the codes, copied ahead from the pages (cp.async, each thread its own 16-byte
//     parts), become fp16 tiles in shared memory (a ring of four, K and V in turn) in the 128-byte swizzle that
//     the tensor core reads: K as a K-major operand, V, whose channels are contiguous, as an
//     MN-major one;
//   * warp 12 issues S, warp 13 P . V.
// P is the A operand from tensor memory, which halves P . V's reading of shared memory.  S has
// one buffer for both tiles in turn, which staggers the two softmax groups by half a step.
//
// Rounding.  P is rounded to fp16 as 2^7 * p * scale_v / 2^w: both are powers of two in the exponent,
// x + log2 scale_v - w, and w is a whole number at most 8 below the row's largest such sum so far (raised
// then, which rescales acc, to the next whole number), so P stays within 2^15 and acc is rescaled rarely.
// Relative error 2^-11; products below 2^-20 of the row's largest are fp16 subnormals.  w is the row's
// own, over the keys that it sees: no block that it does not see, and no other row, changes it.  The sum of
// p is relative to 2^m, m the maximum rounded up: a block's sum of P's exponentials times one power.
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
constexpr int kWarpConvert = 8, kWarpQK = 12, kWarpPV = 13;
constexpr int kStages = 4;  // fp16 tiles
constexpr int kRaw = 2;     // tiles of codes on their way
constexpr int kWindow = 16;  // steps whose scales are in shared memory, two windows in turn for each tile
constexpr uint32_t kTmemCols = 512, kColS = 0;
__host__ __device__ constexpr uint32_t col_p(int t) { return 128u + 64u * uint32_t(t); }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * uint32_t(t); }
constexpr uint32_t kRegsSoftmax = 176, kRegsConvert = 88, kRegsIssue = 72, kLaunchRegs = 128;
static_assert(128 * (2 * kRegsSoftmax + kRegsConvert + kRegsIssue) <= kLaunchRegs * kThreads,
              "the register split must fit the registers the block is launched with");
constexpr float kGrow = 8.0f, kPBits = 7.0f;  // see Rounding above
constexpr uint32_t kMinusInf = 0xff800000u;

constexpr int kBarQFull = 0, kBarKvFull = 2, kBarKvEmpty = kBarKvFull + kStages, kBarSFull = kBarKvEmpty + kStages,
              kBarSEmpty = kBarSFull + 2, kBarPFull = kBarSEmpty + 1, kBarPvDone = kBarPFull + 2,
              kBarOFull = kBarPvDone + 2, kBarOEmpty = kBarOFull + 2, kBarDrain = kBarOEmpty + 2, kNumBars = kBarDrain + 2;

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

__device__ __forceinline__ Reach reach_of(const CacheAttnArgs &A, const Seq &s, int p)
{
    return sa::reach_of(s.n, s.len, A.G, A.causal, A.window, p);
}
__device__ __forceinline__ int64_t steps_of(const CacheAttnArgs &A, const Seq &s, int p0, int stride)
{
    return sa::steps_of(s.n, s.len, A.G, A.causal, A.window, p0, stride);
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

template <int D>
struct Sizes {
    static constexpr int kSub = D / 64;                      // 64-channel halves of a tile
    static constexpr uint32_t kSubBytes = 128 * 128;         // 128 rows x 128 bytes
    static constexpr uint32_t kTileBytes = kSub * kSubBytes; // a Q, K or V tile in fp16
    static constexpr uint32_t kOffQ = 0, kOffKv = 2 * kTileBytes;
    static constexpr uint32_t kRawBytes = 128 * D;
    static constexpr uint32_t kOffRaw = kOffKv + kStages * kTileBytes;
    static constexpr uint32_t kOffScale = kOffRaw + kRaw * kRawBytes;
    static constexpr uint32_t kOffBar = kOffScale + 2 * 2 * 2 * kWindow * 8;
    static constexpr uint32_t kOffWalk = kOffBar + 8 * (kNumBars + 1);
    static constexpr uint32_t kOffMisc = kOffWalk + uint32_t(sizeof(Walk)) * (kWarpPV + 1);
    static constexpr uint32_t kAlloc = kOffMisc + 48;  // range, first, tensor memory's address, abort flag
    static constexpr int kPart = kRowsSeg * (D + 2);
};
static_assert(Sizes<128>::kAlloc <= 227 * 1024, "shared memory per CTA");
static_assert(8 * kCacheChunkMaxSeqs <= kStages * Sizes<64>::kTileBytes, "the costs fit the ring before it is used");

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

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 codes to shared memory, or zeros; a thread waits for its own copies, group by group.
__device__ __forceinline__ void copy_codes(uint32_t dst, const int8_t *src, bool any)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(any ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_f2(uint32_t addr, float a, float b)
{
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
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

// Packed pairs of floats, and in-order forms of the steps below: their relative order is kept as
// written.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(float &a, float &b, uint64_t d)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2_ord(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2_ord(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm volatile("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float ex2_ord(float x)
{
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2_ord(float a, float b)
{
    uint32_t r;
    asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// 32 scores -> 16 words of P, and the sums of 2^(s * c + bias).  Written as a software pipeline
// over groups of four: arguments of group g + 1, ex2 of group g, sums and packing of group g - 1.
__device__ __forceinline__ void p32(const uint32_t (&s)[32], uint64_t c, uint64_t bias, uint64_t (&sum)[2], uint32_t (&pw)[16])
{
    uint64_t y[2][2];
    float e[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) y[0][i] = fma2_ord(pair(fl_of(s[2 * i]), fl_of(s[2 * i + 1])), c, bias);
#pragma unroll
    for (int g = 0; g < 9; ++g) {
        const int cur = g & 1, nxt = cur ^ 1;
        if (g < 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a, b;
                unpair(a, b, y[cur][i]);
                e[cur][2 * i] = ex2_ord(a);
                e[cur][2 * i + 1] = ex2_ord(b);
            }
        }
        if (g + 1 < 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                y[nxt][i] = fma2_ord(pair(fl_of(s[4 * g + 4 + 2 * i]), fl_of(s[4 * g + 5 + 2 * i])), c, bias);
        }
        if (g >= 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] = add2_ord(sum[i], pair(e[nxt][2 * i], e[nxt][2 * i + 1]));
                pw[2 * g - 2 + i] = pack_h2_ord(e[nxt][2 * i], e[nxt][2 * i + 1]);
            }
        }
    }
}
// The same for any mask (unseen keys have the score -inf) and scales: what is not seen is 0 whatever
// the scales.  A row whose sum can be taken from its weights gets the very sums of p32, so that it does
// not depend on the rows that brought its warp here; the others' are those of 2^(s * c - m).
__device__ __forceinline__ void p32_any(const uint32_t (&s)[32], float c, float bias, bool apart, float m, float (&sum)[4],
                                        uint32_t (&pw)[16])
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool seen = s[i + k] != kMinusInf;
            p[k] = seen ? ex2_approx(fmaf(fl_of(s[i + k]), c, bias)) : 0.0f;
            sum[(i & 2) + k] += !apart ? p[k] : seen ? ex2_approx(fmaf(fl_of(s[i + k]), c, -m)) : 0.0f;
        }
        pw[i / 2] = pack_h2(p[0], p[1]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) cache_chunk_kernel(const CacheAttnArgs A)
{
    using S = Sizes<D>;
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128, false), kIdescPV = idesc_f16_f32(128, D, true);
    // All shared memory is dynamic, so that it starts at the 1024-byte boundary that the tiles need.
    extern __shared__ __align__(1024) uint8_t smem[];
    int64_t *range = reinterpret_cast<int64_t *>(smem + S::kOffMisc);   // flattened start, total
    int *first = reinterpret_cast<int *>(smem + S::kOffMisc + 16);      // sequence, head, segment and step of the start
    uint32_t *tmem_word = reinterpret_cast<uint32_t *>(smem + S::kOffMisc + 32);
    int64_t *cost = reinterpret_cast<int64_t *>(smem + S::kOffKv);  // steps of a sequence's segments, of one head
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = reinterpret_cast<int *>(smem + S::kOffMisc + 36);
    if (sbase & 1023u) {  // never so far; the tiles would be read wrongly
        chain_begin();
        if (threadIdx.x == 0) {
            record(6);
            A.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing to join
        }
        return;
    }
    auto bar = [&](int i) -> uint32_t { return sbase + S::kOffBar + 8u * uint32_t(i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar(kBarKvFull + i), 4);
            mbar_init(bar(kBarKvEmpty + i), 1);
        }
        mbar_init(bar(kBarSEmpty), 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(kBarQFull + t), 4);
            mbar_init(bar(kBarSFull + t), 1);
            mbar_init(bar(kBarPFull + t), 4);
            mbar_init(bar(kBarPvDone + t), 1);
            mbar_init(bar(kBarOFull + t), 1);
            mbar_init(bar(kBarOEmpty + t), 4);
            mbar_init(bar(kBarDrain + t), 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpQK) tmem_alloc(smem_u32(tmem_word), kTmemCols);
    chain_begin();
    // ---- the work: a warp sums a sequence's segments, or with many sequences each thread one's
    if (A.B > 64) {
        for (int b = threadIdx.x; b < A.B; b += kThreads) {
            const Seq s = load_seq(A, b);
            cost[b] = steps_of(A, s, 0, 1);
        }
    } else for (int b = warp; b < A.B; b += kThreads / 32) {
        const Seq s = load_seq(A, b);
        int64_t sum = steps_of(A, s, lane, 32);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
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
                const int64_t mine = b + lane < A.B ? cost[b + lane] * A.H : 0;
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
            int64_t rem = (start - before) % cost[b];
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
                first[3] = int(rem);
            }
        }
    }
    __syncthreads();
    const uint32_t tmem = *tmem_word;
    const int64_t total = range[1], chunk = (total + gridDim.x - 1) / gridDim.x;
    Walk &w = reinterpret_cast<Walk *>(smem + S::kOffWalk)[min(warp, kWarpPV)];
    if (lane == 0 && warp <= kWarpPV) {
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
                    if (g == 1 && int(blockIdx.x) == A.quit) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = (2 * g) % kStages;
                    wait(kBarKvFull + st, ((2 * g) / kStages));
                    const uint64_t kd = sdesc(sbase + S::kOffKv + st * S::kTileBytes, 1024, SWZ_128B);
                    for (int t = 0; t < nt && ok; ++t, ++u) {
                        if (u >= 1) wait(kBarSEmpty, (u - 1));
                        if (!ok) break;
                        tc_fence_after();
                        // a step of 16 channels is 32 bytes, 64 channels a half tile; in units of 16
                        const uint64_t qd = sdesc(sbase + S::kOffQ + uint32_t(t) * S::kTileBytes, 1024, SWZ_128B);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t at = uint32_t(kk / 4) * (S::kSubBytes / 16) + uint32_t(kk % 4) * 2;
                                mma_f16(tmem + kColS, qd + at, kd + at, kIdescQK, kk > 0);
                            }
                            tc_commit(bar(kBarSFull + t));
                            if (t == nt - 1) tc_commit(bar(kBarKvEmpty + st));
                        }
                        __syncwarp();
                    }
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
                    const uint64_t vd = sdesc_mn16(sbase + S::kOffKv + st * S::kTileBytes, S::kSubBytes, 1024);
                    for (int t = 0; t < nt && ok; ++t) {
                        wait(kBarPFull + t, c[t]);
                        if (ok && j == 0 && o[t] >= 1) wait(kBarOEmpty + t, (o[t] - 1));
                        if (!ok) break;
                        ++c[t];
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)  // 16 rows of 128 bytes a step
                                mma_f16_ta(tmem + col_o(t), tmem + col_p(t) + 8 * kk, vd + 128 * kk, kIdescPV,
                                           (j > 0 || kk > 0) ? 1u : 0u);
                            tc_commit(bar(kBarPvDone + t));
                            if (j == w.count - 1) tc_commit(bar(kBarOFull + t));
                            if (t == nt - 1) tc_commit(bar(kBarKvEmpty + st));
                        }
                        __syncwarp();
                    }
                }
                for (int t = 0; t < nt; ++t) ++o[t];
            }
        }
        if (!ok && warp <= kWarpPV) {  // the products in flight must land before tensor memory is given up
            if (lane == 0) *abort_flag = 1;
            const uint32_t drain = bar(kBarDrain + warp - kWarpQK);
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            drain_wait(drain, 0);
        }
    } else if (warp >= kWarpConvert) {
        // ---------------------------------------------------------------- codes to fp16 tiles
        regs_dec<kRegsConvert>();
        // A thread takes 16-byte chunks of codes at one channel offset, kPasses of them a tile.  The 16
        // values become two neighbouring 16-byte chunks of a row; eight lanes write two rows of four, so
        // the swizzle spreads a store over all banks.
        constexpr int kRowsPass = 2048 / D;  // rows that the 128 threads take at once
        constexpr int kPasses = 128 / kRowsPass, kHalf = kPasses / 2;
        const int tid = threadIdx.x - 32 * kWarpConvert, wc = tid / 32;
        const int chunk16 = lane % 4 + (D == 128 ? 4 * (wc & 1) : 0);
        const int row = lane / 4 + 8 * (D == 128 ? wc >> 1 : wc);
        const uint32_t to = sbase + S::kOffKv + uint32_t(chunk16 / 4) * S::kSubBytes + uint32_t(row) * 128;
        const uint32_t to0 = to + ((uint32_t(chunk16 % 4 * 2) ^ uint32_t(row & 7)) << 4);
        const uint32_t to1 = to + ((uint32_t(chunk16 % 4 * 2 + 1) ^ uint32_t(row & 7)) << 4);
        const uint32_t raw = sbase + S::kOffRaw + uint32_t(tid) * 16;  // this thread's part of a pass
        uint32_t u = 0;  // tiles
        for (; ok && w.open(A); w.next(A)) {
            // tile i of the piece: K of step i / 2 (i even), or V
            const int tiles = 2 * w.count;
            // lane k: the page of block k of a window of 16 steps, -1 for none; and of the window after
            auto window = [&](int j) {
                const int blk = w.r.blo + 2 * (w.off + j) + lane;
                int page = -1;
                if (blk < w.r.bhi && 2 * j + lane < tiles) {
                    page = A.table[int64_t(w.b) * A.max_pages + blk];
                    if (page < 0 || page >= A.num_pages) {
                        record(8);
                        page = 0;  // its scales are NaN
                    }
                }
                return page;
            };
            const int64_t from = int64_t(w.h) * (kPage * D) + row * D + 16 * chunk16, page_size = int64_t(A.H) * (kPage * D);
            int page_l = window(0), page_n = window(16);
            auto fetch = [&](int i, uint32_t slot) {
                if (i % 32 == 0 && i > 0) {
                    page_l = page_n;
                    page_n = window(i / 2 + 16);
                }
                const int8_t *codes = ((i & 1) ? A.v_codes : A.k_codes) + from;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int page = __shfl_sync(0xffffffffu, page_l, 2 * (i / 2 % 16) + hf);
                    const int8_t *src = codes + max(page, 0) * page_size;
#pragma unroll
                    for (int k = 0; k < kHalf; ++k)
                        copy_codes(raw + slot * S::kRawBytes + (hf * kHalf + k) * 2048, src + k * kRowsPass * D, page >= 0);
                }
                copy_commit();
            };
#pragma unroll 1
            for (int i = 0; i < kRaw; ++i) fetch(i, (u + i) % kRaw);  // a piece has a step at least
#pragma unroll 1
            for (int i = 0; i < tiles; ++i, ++u) {
                const uint32_t st = u % kStages, slot = u % kRaw;
                copy_wait<kRaw - 1>();
                uint4 x[kPasses];
#pragma unroll
                for (int k = 0; k < kPasses; ++k) x[k] = ld_shared_u4(raw + slot * S::kRawBytes + k * 2048);
                if (u >= kStages && !wait(kBarKvEmpty + st, u / kStages - 1)) break;
                const uint32_t at = st * S::kTileBytes;
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const uint32_t wd[4] = {x[k].x ^ 0x80808080u, x[k].y ^ 0x80808080u, x[k].z ^ 0x80808080u,
                                            x[k].w ^ 0x80808080u};
                    st_shared_v4(to0 + at + k * kRowsPass * 128,
                                 make_uint4(bytes_to_h2(wd[0], 0x4140u), bytes_to_h2(wd[0], 0x4342u),
                                            bytes_to_h2(wd[1], 0x4140u), bytes_to_h2(wd[1], 0x4342u)));
                    st_shared_v4(to1 + at + k * kRowsPass * 128,
                                 make_uint4(bytes_to_h2(wd[2], 0x4140u), bytes_to_h2(wd[2], 0x4342u),
                                            bytes_to_h2(wd[3], 0x4140u), bytes_to_h2(wd[3], 0x4342u)));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarKvFull + st));
                // the parts just read are this thread's own, so they may be written again
                if (i + kRaw < tiles)
                    fetch(i + kRaw, slot);
                else
                    copy_commit();
            }
        }
        copy_wait<0>();
    } else {
        // ---------------------------------------------------------------- softmax of tile t
        regs_inc<kRegsSoftmax>();
        const int t = warp >> 2, wq = warp & 3;
        const int row = wq * 32 + lane;
        const uint32_t lane_addr = uint32_t(wq * 32) << 16;
        uint32_t turn = 0;  // windows of scales so far
        uint32_t c = 0, o = 0;  // steps and pieces of this tile
        bool split = false;
        const int wk = int(blockIdx.x);
        for (; w.open(A); w.next(A)) {
            if (t >= w.tiles(A)) continue;
            int lo, hi;  // the keys that this row sees, [lo, hi); rows past the last see all, and are not written
            {
                const int rr = w.p * kRowsSeg + t * 128 + row, pos = w.s.len - w.s.n + rr / A.G;
                const bool valid = rr < w.s.n * A.G;
                hi = min(valid && (A.causal || pos < 0) ? pos + 1 : w.s.len, w.r.bhi * kPage);
                lo = valid && A.window > 0 ? max(0, pos - A.window + 1) : 0;
            }
            // The scales are found a window of 16 steps at a time, the pages two windows and the scales one
            // ahead; lane i has those of block i of the window.
            auto page_at = [&](int j) {  // -1: no such block
                const int blk = w.r.blo + 2 * (w.off + j) + lane;
                return blk < w.r.bhi && 2 * j + lane < 2 * w.count ? A.table[int64_t(w.b) * A.max_pages + blk] : -1;
            };
            auto scales_at = [&](int j, int page, float &sk, float &sv) {
                const int blk = w.r.blo + 2 * (w.off + j) + lane;
                sk = sv = 0.0f;
                if (!(blk < w.r.bhi && 2 * j + lane < 2 * w.count)) return;
                sk = sv = __int_as_float(0x7fffffff);
                if (page < 0 || page >= A.num_pages) return;
                sk = A.k_scale[int64_t(page) * A.H + w.h];
                sv = A.v_scale[int64_t(page) * A.H + w.h];
            };
            int page_n = page_at(0);
            // ---- the rows of q, fp16 (the tile is free: S of the last step before was read).  A row takes kLanes
            // lanes, 16 bytes each; all loads are in flight at once.
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
            float rc, sk_n, sv_n;
            {
                const int rr = w.p * kRowsSeg + t * 128 + row, i = rr / A.G;
                const int64_t own = rr < w.s.n * A.G ? (int64_t(w.s.ts) + i) * A.q_stride + int64_t(w.h * A.G + rr - i * A.G) * D : -1;
                uint4 x[kLanes];
#pragma unroll
                for (int k = 0; k < kLanes; ++k) {
                    const int64_t from = __shfl_sync(0xffffffffu, own, k * kAtOnce + lane / kLanes);
                    x[k] = make_uint4(0, 0, 0, 0);
                    if (from >= 0)
                        x[k] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(A.q) + from + 8 * (lane % kLanes));
                }
                scales_at(0, page_n, sk_n, sv_n);
                page_n = page_at(kWindow);
                uint32_t mine = 0;  // bits of the largest |q| of this thread's row
#pragma unroll
                for (int k = 0; k < kLanes; ++k) {
                    const int r = wq * 32 + k * kAtOnce + lane / kLanes, chunk = lane % kLanes;
                    uint4 v = x[k];
                    if (A.dtype == 0) {
                        uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
#pragma unroll
                        for (int o = 1; o < kLanes; o *= 2) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                        top = max(top & 0xffffu, top >> 16);
                        const uint32_t theirs = __shfl_sync(0xffffffffu, top, lane % kAtOnce * kLanes);
                        mine = lane / kAtOnce == k ? theirs : mine;
                        float up, down;
                        row_power(__uint_as_float(top << 16), up, down);
                        uint32_t *w4 = &v.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w4[e] = pack_h2(__uint_as_float(w4[e] << 16) * up, __uint_as_float(w4[e] & 0xffff0000u) * up);
                    }
                    st_shared_v4(sbase + S::kOffQ + uint32_t(t) * S::kTileBytes + (chunk / 8) * S::kSubBytes + r * 128 +
                                     (((chunk & 7) ^ (r & 7)) << 4),
                                 v);
                }
                float up, down = 1.0f;
                if (A.dtype == 0) row_power(__uint_as_float(mine << 16), up, down);
                rc = A.sm_scale * kLog2e * down;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarQFull + t));
            }
            float m = -INFINITY, l = 0.0f, w_ref = -INFINITY;
            // The scales go to shared memory, for each block scale_k and log2 scale_v.  The four warps
            // of the tile write the same values, two windows in turn: none is further than into its next
            // window while another reads the one before, for each S needs all four to have read the last.
            uint32_t scales = 0;
            for (int j = 0; j < w.count; ++j, ++c) {
                if (j % kWindow == 0) {
                    scales = sbase + S::kOffScale + uint32_t(2 * t + (turn++ & 1)) * (2 * kWindow * 8);
                    const int blk = w.r.blo + 2 * (w.off + j) + lane;
                    if (blk < w.r.bhi)
                        st_shared_f2(scales + 8 * lane, sk_n, log2_scale(sv_n));
                    else
                        st_shared_f2(scales + 8 * lane, 1.0f, 0.0f);  // no such block: none of its keys is seen
                    __syncwarp();
                    scales_at(j + kWindow, page_n, sk_n, sv_n);
                    page_n = page_at(j + 2 * kWindow);
                }
                const int t0 = (w.r.blo + 2 * (w.off + j)) * kPage;
                const bool edge = __any_sync(0xffffffffu, lo > t0 || hi < t0 + 2 * kPage);
                const float4 b = ld_shared_f4(scales + 16 * (j % kWindow));  // of both blocks
                const float c0 = rc * b.x, c1 = rc * b.z;
                if (!wait(kBarSFull + t, c)) break;
                uint32_t s[4][32];
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32_nowait(tmem + lane_addr + kColS + 32 * k, s[k]);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k) regs_ready(s[k]);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int first = lo - (t0 + 32 * k), end = hi - (t0 + 32 * k);
                        if (!__any_sync(0xffffffffu, first > 0 || end < 32)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e < first || e >= end) s[k][e] = kMinusInf;
                    }
                }
                // the scales are not negative, so they commute with the maximum (0 * -inf is
                // a NaN, which fmaxf passes over)
                const float top0 = max64(s[0], s[1]) * c0, top1 = max64(s[2], s[3]) * c1;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarSEmpty));

                const float top = fmaxf(top0, top1), most = fmaxf(top0 + b.y, top1 + b.w);
                float f = 1.0f;  // what acc is rescaled by
                if (top > m) {
                    const float up = ceilf(top);
                    l *= ex2_approx(m - up);
                    m = up;
                }
                if (most > w_ref + kGrow || (w_ref == -INFINITY && most > w_ref)) {
                    const float up = ceilf(most);
                    f = ex2_approx(w_ref - up);
                    w_ref = up;
                }
                // bias: P = 2^(x + bias); at: the exponent of P at x = m
                const float ref = m == -INFINITY ? 0.0f : m, base = kPBits - (w_ref == -INFINITY ? 0.0f : w_ref);
                const float bias0 = base + b.y, bias1 = base + b.w, at0 = bias0 + ref, at1 = bias1 + ref;
                // else P may vanish where p does not, and unseen keys need more than a score of -inf
                const bool plain0 = at0 >= kAtLeast && c0 > 0.0f && c0 < INFINITY;
                const bool plain1 = at1 >= kAtLeast && c1 > 0.0f && c1 < INFINITY;
                const bool plain = __all_sync(0xffffffffu, plain0 && plain1);
                // P's columns and acc are free once P . V of the step before is done
                if (c >= 1 && !wait(kBarPvDone + t, c - 1)) break;
                tc_fence_after();
                if (plain) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pw[16];
                        uint64_t sum[2] = {0, 0};
                        const float cc = k < 2 ? c0 : c1, bias = k < 2 ? bias0 : bias1;
                        p32(s[k], pair(cc, cc), pair(bias, bias), sum, pw);
                        tmem_st16(tmem + lane_addr + col_p(t) + 16 * k, pw);
                        float x0, x1, x2, x3;
                        unpair(x0, x1, sum[0]);
                        unpair(x2, x3, sum[1]);
                        l = fmaf((x0 + x1) + (x2 + x3), ex2_approx(k < 2 ? -at0 : -at1), l);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pw[16];
                        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        const bool apart = !(k < 2 ? plain0 : plain1);
                        p32_any(s[k], k < 2 ? c0 : c1, k < 2 ? bias0 : bias1, apart, ref, sum, pw);
                        tmem_st16(tmem + lane_addr + col_p(t) + 16 * k, pw);
                        l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), apart ? 1.0f : ex2_approx(k < 2 ? -at0 : -at1), l);
                    }
                }
                if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t r[32];
                        tmem_ld32_wait(tmem + lane_addr + col_o(t) + 32 * k, r);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float x, y;
                            mul2(x, y, fl_of(r[e]), fl_of(r[e + 1]), f, f);
                            r[e] = __float_as_uint(x);
                            r[e + 1] = __float_as_uint(y);
                        }
                        tmem_st32(tmem + lane_addr + col_o(t) + 32 * k, r);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarPFull + t));
            }
            // ---- epilogue of the piece
            if (!ok || !wait(kBarOFull + t, o)) break;
            {
                tc_fence_after();
                const int rr = w.p * kRowsSeg + t * 128 + row, i = rr / A.G;
                const bool valid = rr < w.s.n * A.G;
                const int64_t at = (int64_t(w.s.ts) + i) * (A.H * A.G) + w.h * A.G + rr - i * A.G;
                const bool whole = w.begins && w.ends;
                const int slot = 2 * wk + (w.pieces == 0 ? 0 : 1);
                float f, power;
                power_of(w_ref, m, kPBits, f, power);
                if (whole) f = l == 0.0f ? 0.0f : f / l;
                float *part = A.part + int64_t(slot) * S::kPart;
                if (w.begins && !w.ends) {
                    split = true;
                    if (t == 0 && wq == 0 && lane == 0) {
                        A.meta[2 * wk] = make_int4(int((w.pos + w.r.steps() - 1) / chunk) - wk + 1, slot, 0, 0);
                        A.meta[2 * wk + 1] = make_int4(w.s.ts, w.h, w.p * kRowsSeg, min(kRowsSeg, w.s.n * A.G - w.p * kRowsSeg));
                    }
                }
                if (valid && whole && A.lse) A.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                if (valid && !whole) {
                    part[kRowsSeg * D + t * 128 + row] = m;
                    part[kRowsSeg * (D + 1) + t * 128 + row] = l;
                }
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t r[32];
                    tmem_ld32_wait(tmem + lane_addr + col_o(t) + 32 * k, r);
                    if (!valid) continue;
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(fl_of(r[e]) * f * power);
                    if (whole) {
                        T *dst = static_cast<T *>(A.o) + at * D + 32 * k;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(dst + e) =
                                make_uint4(pack_out(fl_of(r[e]), fl_of(r[e + 1]), T()),
                                           pack_out(fl_of(r[e + 2]), fl_of(r[e + 3]), T()),
                                           pack_out(fl_of(r[e + 4]), fl_of(r[e + 5]), T()),
                                           pack_out(fl_of(r[e + 6]), fl_of(r[e + 7]), T()));
                    } else {
                        float *dst = part + (8 * k * kRowsSeg + t * 128 + row) * 4;  // [D / 4][row][4]
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + e * kRowsSeg) =
                                make_float4(fl_of(r[e]), fl_of(r[e + 1]), fl_of(r[e + 2]), fl_of(r[e + 3]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarOEmpty + t));
            ++o;
        }
        // tile A takes part in every piece, so it knows whether a segment was begun and not ended
        if (warp == 0 && lane == 0 && !split) A.meta[2 * wk] = make_int4(0, 0, 0, 0);
    }
    if (lane == 0 && !ok) {
        *abort_flag = 1;
        record(6);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpQK) tmem_dealloc(tmem, kTmemCols);
    if (*abort_flag) {  // what others join with this block's pieces is to be NaN, whichever of them it wrote
        static_assert(2 * kRowsSeg == kThreads, "a maximum for each thread");
        A.part[int64_t(2 * blockIdx.x + threadIdx.x / kRowsSeg) * S::kPart + kRowsSeg * D + threadIdx.x % kRowsSeg] =
            __int_as_float(0x7fffffff);
    }
}

// Joins the pieces of the segment that worker blockIdx.x began and others went on with, in the
// order of the workers.  A piece is acc [D / 4][256][4], m [256], l [256]: a warp takes 32 rows, one
// a lane, and 16 channels, so its reads are contiguous.
constexpr int kCombineThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) cache_chunk_combine_kernel(const CacheAttnArgs A)
{
    constexpr int kPart = Sizes<D>::kPart, kGroups = kRowsSeg / 32;
    chain_begin();
    const int w = blockIdx.x, task = blockIdx.y * (kCombineThreads / 32) + (threadIdx.x >> 5);
    const int4 meta = A.meta[2 * w], where = A.meta[2 * w + 1];
    const int row = task % kGroups * 32 + (threadIdx.x & 31), ch = task / kGroups * 16;
    if (meta.x == 0 || row >= where.w) return;
    auto part_of = [&](int p) { return A.part + int64_t(p == 0 ? meta.y : 2 * (w + p)) * kPart; };
    float big = -INFINITY, total = 0.0f, out[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) out[e] = 0.0f;
#pragma unroll 4
    for (int p = 0; p < meta.x; ++p) big = fmaxf(big, part_of(p)[kRowsSeg * D + row]);
    const float ref = big == -INFINITY ? 0.0f : big;
#pragma unroll 2
    for (int p = 0; p < meta.x; ++p) {
        const float *part = part_of(p);
        const float f = ex2_approx(part[kRowsSeg * D + row] - ref);
        total = fmaf(f, part[kRowsSeg * (D + 1) + row], total);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(part + ((ch + e) / 4 * kRowsSeg + row) * 4);
            out[e] = fmaf(f, v.x, out[e]);
            out[e + 1] = fmaf(f, v.y, out[e + 1]);
            out[e + 2] = fmaf(f, v.z, out[e + 2]);
            out[e + 3] = fmaf(f, v.w, out[e + 3]);
        }
    }
    const float f = total == 0.0f ? 0.0f : 1.0f / total;
    const int rr = where.z + row, i = rr / A.G;
    const int64_t at = (int64_t(where.x) + i) * (A.H * A.G) + where.y * A.G + rr - i * A.G;
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = pack_out(out[2 * e] * f, out[2 * e + 1] * f, T());
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(A.o) + at * D + ch);
    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
    if (A.lse && ch == 0) A.lse[at] = total == 0.0f ? -INFINITY : (big + log2f(total)) * kLn2;
}

template <typename T, int D>
cudaError_t launch_for(const CacheAttnArgs &a, int sms, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(cache_chunk_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(Sizes<D>::kAlloc));
    if (e != cudaSuccess) return e;
    e = launch_chained(cache_chunk_kernel<T, D>, dim3(unsigned(sms)), kThreads, Sizes<D>::kAlloc, st, a);
    if (e != cudaSuccess) return e;
    return launch_chained(cache_chunk_combine_kernel<T, D>, dim3(unsigned(sms), D / 16), kCombineThreads, 0, st, a);
}

}  // namespace

size_t cache_chunk_part_bytes(int sms, int d)
{
    return size_t(2) * sms * size_t(d == 128 ? Sizes<128>::kPart : Sizes<64>::kPart) * 4;
}

cudaError_t launch_cache_chunk(const CacheAttnArgs &a, int sms, cudaStream_t st)
{
    if (a.dtype == 0)
        return a.d == 128 ? launch_for<__nv_bfloat16, 128>(a, sms, st)
                          : launch_for<__nv_bfloat16, 64>(a, sms, st);
    return a.d == 128 ? launch_for<__half, 128>(a, sms, st) : launch_for<__half, 64>(a, sms, st);
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
