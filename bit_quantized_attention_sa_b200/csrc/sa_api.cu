// sa_api.cu -- the C ABI declared in include/sa.h: argument validation, the per-device
// grow-only workspace, TMA tensor-map encoding and launch sequencing on the caller's
// stream.  No entry point synchronises except sa_get_device_status and
// sa_release_workspace.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <numeric>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/sa.h"
#include "sa_cache_attn.cuh"
#include "sa_internal.h"

namespace sa {

// ------------------------------------------------------------------ tensor maps

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

bool encode_tmap_2d_u8(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                       uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                       CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {row_stride_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tmap_3d_f32(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                        uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1,
                        CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
    const cuuint32_t box[3] = {box0, box1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device's SM count (0: no device), asked for once per device.
int device_sms()
{
    static std::atomic<int> cached[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64 && (sms = cached[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) cached[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// ------------------------------------------------------------------ validation

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static sa_status check_shape(int B, int H, int N, int d, Shape *s)
{
    if (B < 1 || H < 1 || N < 1) return SA_ERR_INVALID_ARG;
    if (d != kD) return SA_ERR_UNSUPPORTED;
    s->B = B;
    s->H = H;
    s->N = N;
    // TMA row coordinates and tile indices are 32-bit
    if (s->BH() > INT_MAX / 8 || s->BH() * s->Npad() > INT_MAX) return SA_ERR_INVALID_ARG;
    // the heads are a grid dimension (y) of the prologue kernels
    if (s->BH() > 65535) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

static sa_status check_ptrs(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if (!p) return SA_ERR_INVALID_ARG;
    for (const void *p : ps)
        if (!aligned16(p)) return SA_ERR_MISALIGNED;
    return SA_OK;
}

// sm_100 device check, cached per device.
static sa_status check_device()
{
    static int cached[64];  // 0 unknown, 1 ok, 2 unsupported
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SA_ERR_CUDA;
    if (dev >= 0 && dev < 64 && cached[dev]) return cached[dev] == 1 ? SA_OK : SA_ERR_UNSUPPORTED;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return SA_ERR_CUDA;
    const bool ok = (major == 10 && minor == 0);
    if (dev >= 0 && dev < 64) cached[dev] = ok ? 1 : 2;
    return ok ? SA_OK : SA_ERR_UNSUPPORTED;
}

// ------------------------------------------------------------------ workspace

struct WsLayout {
    size_t q8, k8, v8, sq, sk, sv, kmean, kpart, vamax, total;
};

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

static WsLayout ws_layout(const Shape &s)
{
    WsLayout L;
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
    const size_t BH = size_t(s.BH()), Np = size_t(s.Npad());
    L.q8 = take(BH * Np * kD);
    L.k8 = take(BH * Np * kD);
    L.v8 = take(BH * Np * kD);
    L.sq = take(BH * size_t(s.nq()) * 4);
    L.sk = take(BH * size_t(s.nk()) * 4);
    L.sv = take(BH * kD * 4);
    L.kmean = take(BH * kD * 4);
    L.kpart = take(BH * size_t(s.nchunks()) * kD * 8);
    L.vamax = take(BH * kD * 4);
    L.total = off;
    return L;
}

struct DeviceWs {
    void *ptr = nullptr;
    size_t bytes = 0;
};
static DeviceWs g_ws[64];
// Held by a call from its workspace request until its launches are enqueued, so that no
// other host thread can grow (and so free) the buffer in between.  Recursive: the d = 64
// and SLA paths request the workspace again inside the same call.
static std::recursive_mutex g_ws_mutex;
typedef std::unique_lock<std::recursive_mutex> WsLock;

// Returns the current device's workspace grown to at least `bytes`, with `lock` held.
static sa_status get_workspace(WsLock &lock, size_t bytes, uint8_t **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SA_ERR_CUDA;
    if (!lock.owns_lock()) lock = WsLock(g_ws_mutex);
    DeviceWs &w = g_ws[dev];
    if (w.bytes < bytes) {
        if (w.ptr) {
            // work enqueued earlier, on any stream, may still use the old buffer
            if (cudaDeviceSynchronize() != cudaSuccess) return SA_ERR_CUDA;
            cudaFree(w.ptr);
            w.ptr = nullptr;
            w.bytes = 0;
        }
        if (cudaMalloc(&w.ptr, bytes) != cudaSuccess) {
            cudaGetLastError();
            w.ptr = nullptr;
            return SA_ERR_OOM;
        }
        w.bytes = bytes;
    }
    *out = static_cast<uint8_t *>(w.ptr);
    return SA_OK;
}

// Page-locked host staging for small tables that a call uploads (variable-length
// batches), per device, grow-only.  Used with the workspace lock held; the event marks the
// last upload, which must have left the buffer before it is overwritten.
struct HostStage {
    void *ptr = nullptr;
    size_t bytes = 0;
    cudaEvent_t ev = nullptr;
};
static HostStage g_stage[64];

static sa_status upload_table(const void *src, size_t n, void *dst, cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SA_ERR_CUDA;
    HostStage &h = g_stage[dev];
    if (!h.ev) {
        if (cudaEventCreateWithFlags(&h.ev, cudaEventDisableTiming) != cudaSuccess) return SA_ERR_CUDA;
    } else if (cudaEventSynchronize(h.ev) != cudaSuccess) {
        return SA_ERR_CUDA;
    }
    if (h.bytes < n) {
        if (h.ptr) cudaFreeHost(h.ptr);
        h.ptr = nullptr;
        h.bytes = 0;
        if (cudaMallocHost(&h.ptr, n) != cudaSuccess) {
            cudaGetLastError();
            return SA_ERR_OOM;
        }
        h.bytes = n;
    }
    std::memcpy(h.ptr, src, n);
    if (cudaMemcpyAsync(dst, h.ptr, n, cudaMemcpyHostToDevice, st) != cudaSuccess) return SA_ERR_CUDA;
    return cudaEventRecord(h.ev, st) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

static sa_status attention_core(const int8_t *q8, const float *sq, const int8_t *k8,
                                const float *sk, const uint8_t *v8, const float *sv, void *o,
                                const Shape &s, float sm_scale, const uint8_t *mask,
                                cudaStream_t st, bool causal = false, const float *addend = nullptr,
                                const SeqTable &seq = SeqTable())
{
    AttnArgs a;
    const uint64_t rows = uint64_t(s.BH() * s.Npad());
    if (!encode_tmap_2d_u8(&a.tm_q, q8, kD, rows, kD, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d_u8(&a.tm_k, k8, kD, rows, kD, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d_u8(&a.tm_v, v8, uint64_t(s.Npad()), uint64_t(s.BH()) * kD,
                           uint64_t(s.Npad()), 64, 128, CU_TENSOR_MAP_SWIZZLE_64B))
        return SA_ERR_CUDA;
    a.q_scale = sq;
    a.k_scale = sk;
    a.v_scale = sv;
    a.mask = mask;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.BH = int(s.BH());
    a.N = int(s.N);
    a.Npad = int(s.Npad());
    a.nq = int(s.nq());
    a.nk = int(s.nk());
    a.sm_scale = sm_scale;
    a.causal = causal ? 1 : 0;
    a.addend = addend;
    a.seq = seq;
    return launch_attention(a, st) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

// Prologue into the library workspace, then the fused attention kernel (validated args).
static sa_status attn_fwd_device(const void *q, const void *k, const void *v, void *o,
                                 const Shape &s, float sm_scale, const uint8_t *block_mask,
                                 cudaStream_t st, bool causal = false, const float *addend = nullptr,
                                 const SeqTable &seq = SeqTable())
{
    const WsLayout L = ws_layout(s);
    WsLock lock;
    uint8_t *ws = nullptr;
    sa_status r = get_workspace(lock, L.total, &ws);
    if (r != SA_OK) return r;
    int8_t *q8 = reinterpret_cast<int8_t *>(ws + L.q8);
    int8_t *k8 = reinterpret_cast<int8_t *>(ws + L.k8);
    uint8_t *v8 = ws + L.v8;
    float *sq = reinterpret_cast<float *>(ws + L.sq);
    float *sk = reinterpret_cast<float *>(ws + L.sk);
    float *sv = reinterpret_cast<float *>(ws + L.sv);
    if (launch_quantize_qk(q, k, s, q8, sq, k8, sk, reinterpret_cast<float *>(ws + L.kmean),
                           reinterpret_cast<double *>(ws + L.kpart), st, seq) != cudaSuccess)
        return SA_ERR_CUDA;
    if (launch_quantize_v(v, s, v8, sv, reinterpret_cast<uint32_t *>(ws + L.vamax), st, seq) !=
        cudaSuccess)
        return SA_ERR_CUDA;
    return attention_core(q8, sq, k8, sk, v8, sv, o, s, sm_scale, block_mask, st, causal, addend, seq);
}

// ------------------------------------------------------------------ host-buffer pipeline
//
// sa_attn_fwd_host: the heads (b, h) are independent, so the B*H heads are cut into chunks
// of consecutive heads; the upload of chunk c+1 and the download of chunk c-1 run on two
// library streams while chunk c is computed on the caller's stream.  Chunk c holds at most
// c + 1 heads (then the full chunk size): the first upload, which nothing overlaps, stays
// one head long, and each later upload still fits under the computation before it.  Two staging slots per
// device alternate between chunks; events order each slot's reuse:
//   upload(c)   waits compute(c-2)   (its inputs were read)
//   compute(c)  waits upload(c) and download(c-2) (its output slot was copied out)
//   download(c) waits compute(c)
// and the caller's stream finally waits for both slots' last download.

constexpr size_t kHostChunkTensorBytes = size_t(64) << 20;  // target bytes of q per chunk

struct HostPipe {
    cudaStream_t h2d = nullptr, d2h = nullptr;
    cudaEvent_t entry = nullptr, in[2] = {nullptr, nullptr}, comp[2] = {nullptr, nullptr},
                out[2] = {nullptr, nullptr};
    void *buf = nullptr;
    size_t bytes = 0;
};
static HostPipe g_hp[64];
static std::mutex g_hp_mutex;

static sa_status host_pipe_init(HostPipe &P)
{
    if (P.h2d) return SA_OK;
    if (cudaStreamCreateWithFlags(&P.h2d, cudaStreamNonBlocking) != cudaSuccess ||
        cudaStreamCreateWithFlags(&P.d2h, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&P.entry, cudaEventDisableTiming) != cudaSuccess)
        return SA_ERR_CUDA;
    for (int i = 0; i < 2; ++i)
        if (cudaEventCreateWithFlags(&P.in[i], cudaEventDisableTiming) != cudaSuccess ||
            cudaEventCreateWithFlags(&P.comp[i], cudaEventDisableTiming) != cudaSuccess ||
            cudaEventCreateWithFlags(&P.out[i], cudaEventDisableTiming) != cudaSuccess)
            return SA_ERR_CUDA;
    return SA_OK;
}

static sa_status attn_fwd_host_pipeline(const void *q, const void *k, const void *v, void *o,
                                        const Shape &s, float sm_scale, const uint8_t *mask,
                                        cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_hp_mutex);
    HostPipe &P = g_hp[dev];
    sa_status r = host_pipe_init(P);
    if (r != SA_OK) return r;

    const int64_t BH = s.BH();
    const size_t head_bytes = size_t(s.N) * kD * 2;                  // one head of q (bf16)
    const size_t head_mask = size_t(s.nq()) * size_t(s.nk());        // one head of the mask
    const int64_t hc = std::max<int64_t>(1, std::min<int64_t>(BH, int64_t(kHostChunkTensorBytes / head_bytes)));
    const size_t t_bytes = align256(size_t(hc) * head_bytes);
    const size_t m_bytes = mask ? align256(size_t(hc) * head_mask) : 0;
    const size_t slot = 4 * t_bytes + m_bytes;
    if (P.bytes < 2 * slot) {
        if (P.buf) {
            // earlier calls may still use the old staging buffer
            if (cudaDeviceSynchronize() != cudaSuccess) return SA_ERR_CUDA;
            cudaFree(P.buf);
            P.buf = nullptr;
            P.bytes = 0;
        }
        if (cudaMalloc(&P.buf, 2 * slot) != cudaSuccess) {
            cudaGetLastError();
            return SA_ERR_OOM;
        }
        P.bytes = 2 * slot;
    }
    const uint8_t *hq = static_cast<const uint8_t *>(q), *hk = static_cast<const uint8_t *>(k),
                  *hv = static_cast<const uint8_t *>(v);
    uint8_t *ho = static_cast<uint8_t *>(o);
    // the inputs may be written by work already enqueued on the caller's stream
    if (cudaEventRecord(P.entry, st) != cudaSuccess || cudaStreamWaitEvent(P.h2d, P.entry, 0) != cudaSuccess)
        return SA_ERR_CUDA;
    int last[2] = {0, 0};
    for (int64_t h0 = 0, c = 0, hn = 0; h0 < BH; h0 += hn, ++c) {
        const int i = int(c & 1);
        hn = std::min<int64_t>(std::min<int64_t>(hc, c + 1), BH - h0);
        const size_t nb = size_t(hn) * head_bytes, off = size_t(h0) * head_bytes;
        uint8_t *base = static_cast<uint8_t *>(P.buf) + size_t(i) * slot;
        uint8_t *dq = base, *dk = base + t_bytes, *dv = base + 2 * t_bytes, *dout = base + 3 * t_bytes;
        uint8_t *dm = mask ? base + 4 * t_bytes : nullptr;
        bool ok = cudaStreamWaitEvent(P.h2d, P.comp[i], 0) == cudaSuccess &&
                  cudaMemcpyAsync(dq, hq + off, nb, cudaMemcpyHostToDevice, P.h2d) == cudaSuccess &&
                  cudaMemcpyAsync(dk, hk + off, nb, cudaMemcpyHostToDevice, P.h2d) == cudaSuccess &&
                  cudaMemcpyAsync(dv, hv + off, nb, cudaMemcpyHostToDevice, P.h2d) == cudaSuccess &&
                  (!mask || cudaMemcpyAsync(dm, mask + size_t(h0) * head_mask, size_t(hn) * head_mask,
                                            cudaMemcpyHostToDevice, P.h2d) == cudaSuccess) &&
                  cudaEventRecord(P.in[i], P.h2d) == cudaSuccess &&
                  cudaStreamWaitEvent(st, P.in[i], 0) == cudaSuccess &&
                  cudaStreamWaitEvent(st, P.out[i], 0) == cudaSuccess;
        if (!ok) return SA_ERR_CUDA;
        Shape sc;
        sc.B = 1;
        sc.H = int(hn);
        sc.N = s.N;
        r = attn_fwd_device(dq, dk, dv, dout, sc, sm_scale, dm, st);
        if (r != SA_OK) return r;
        ok = cudaEventRecord(P.comp[i], st) == cudaSuccess &&
             cudaStreamWaitEvent(P.d2h, P.comp[i], 0) == cudaSuccess &&
             cudaMemcpyAsync(ho + off, dout, nb, cudaMemcpyDeviceToHost, P.d2h) == cudaSuccess &&
             cudaEventRecord(P.out[i], P.d2h) == cudaSuccess;
        if (!ok) return SA_ERR_CUDA;
        last[i] = 1;
    }
    // the call is complete on the caller's stream once the outputs are in host memory
    for (int i = 0; i < 2; ++i)
        if (last[i] && cudaStreamWaitEvent(st, P.out[i], 0) != cudaSuccess) return SA_ERR_CUDA;
    return SA_OK;
}

// Variable-length groups: sequences taken longest first (ord, a stable order); a group
// runs as one prologue and one attention launch over heads padded to its longest sequence,
// and takes the next sequence while the padded size stays within twice the group's own
// (or below 2^20 padded token-heads, where the padding costs little) and its heads stay a
// valid grid dimension.
struct VarlenGroup {
    int first, count;  // positions in ord
    int64_t nmax;
};
static void varlen_groups(int nseq, const int *seqlens, int H, std::vector<int> &ord, std::vector<VarlenGroup> &groups)
{
    ord.resize(static_cast<size_t>(nseq));
    std::iota(ord.begin(), ord.end(), 0);
    std::stable_sort(ord.begin(), ord.end(), [&](int a, int b) { return seqlens[a] > seqlens[b]; });
    groups.clear();
    for (int g0 = 0; g0 < nseq;) {
        const int64_t nmax = seqlens[ord[g0]], pmax = padded_len(nmax);
        int64_t own = pmax;
        int cnt = 1;
        while (g0 + cnt < nseq) {
            const int64_t own2 = own + padded_len(seqlens[ord[g0 + cnt]]), pad2 = int64_t(cnt + 1) * pmax;
            if (pad2 > 2 * own2 && pad2 * H > (int64_t(1) << 20)) break;
            if (int64_t(cnt + 1) * H > 65535) break;
            own = own2;
            ++cnt;
        }
        groups.push_back({g0, cnt, nmax});
        g0 += cnt;
    }
}

// ------------------------------------------------------------------ cache calls

static bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The sizes of a call on the cache.
static sa_status check_cache_sizes(int64_t T, int B, int H, int d)
{
    if (T < 0 || B < 1 || H < 1) return SA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return SA_ERR_UNSUPPORTED;
    if (T > (1 << 30) || B > (1 << 20) || H > 65535 || (T / kPage + 2 * int64_t(B)) * H > INT_MAX) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

// What the calls on the cache share: sizes, the cache's and the sequences' arrays.
static sa_status check_cache(int64_t T, int B, int H, int d, int max_pages, int num_pages, const void *tok_start,
                             const void *kv_lens, const void *table, const void *k_codes, const void *k_scale,
                             const void *v_codes, const void *v_scale)
{
    if (max_pages < 1 || num_pages < 1) return SA_ERR_INVALID_ARG;
    const sa_status r = check_cache_sizes(T, B, H, d);
    if (r != SA_OK) return r;
    // lines of 128 bytes are a 32-bit TMA coordinate; positions and grid dimensions likewise
    if (max_pages > (1 << 30) / kPage || int64_t(num_pages) * H > (int64_t(INT_MAX) * 2) / d) return SA_ERR_UNSUPPORTED;
    if (T == 0) return SA_OK;
    for (const void *p : {tok_start, kv_lens, table, k_codes, k_scale, v_codes, v_scale})
        if (!p) return SA_ERR_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(v_codes)) return SA_ERR_MISALIGNED;
    for (const void *p : {tok_start, kv_lens, table, k_scale, v_scale})
        if (!aligned(p, 4)) return SA_ERR_MISALIGNED;
    return SA_OK;
}

// A packed token tensor whose tokens have `width` values of 16 bits.
static sa_status check_tokens(const void *p, int64_t stride, int64_t width)
{
    if (!p || stride < width) return SA_ERR_INVALID_ARG;
    if (!aligned16(p) || stride % 8 != 0) return SA_ERR_MISALIGNED;
    return SA_OK;
}

}  // namespace sa

using namespace sa;

extern "C" {

sa_status sa_quantize_qk(const void *q, const void *k, int B, int H, int N, int d,
                         int8_t *q_i8, float *q_scale, int8_t *k_i8, float *k_scale,
                         float *k_mean, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({q, k, q_i8, q_scale, k_i8, k_scale, k_mean})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    const WsLayout L = ws_layout(s);
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, L.total, &ws)) != SA_OK) return r;
    cudaError_t e = launch_quantize_qk(q, k, s, q_i8, q_scale, k_i8, k_scale, k_mean,
                                       reinterpret_cast<double *>(ws + L.kpart),
                                       static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_quantize_qk_noalloc(const void *q, const void *k, int B, int H, int N, int d,
                                 int8_t *q_i8, float *q_scale, int8_t *k_i8, float *k_scale,
                                 float *k_mean, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({q, k, q_i8, q_scale, k_i8, k_scale, k_mean})) != SA_OK) return r;
    if (size_t(s.BH()) * size_t(s.nchunks()) * kD > kNoAllocPartialDoubles) return SA_ERR_SCRATCH_LIMIT;
    if ((r = check_device()) != SA_OK) return r;
    double *part = nullptr;
    if (noalloc_kpart(&part) != cudaSuccess) return SA_ERR_CUDA;
    cudaError_t e = launch_quantize_qk(q, k, s, q_i8, q_scale, k_i8, k_scale, k_mean, part,
                                       static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_quantize_v(const void *v, int B, int H, int N, int d, uint8_t *v_fp8_t,
                        float *v_scale, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({v, v_fp8_t, v_scale})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    const WsLayout L = ws_layout(s);
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, L.total, &ws)) != SA_OK) return r;
    cudaError_t e = launch_quantize_v(v, s, v_fp8_t, v_scale,
                                      reinterpret_cast<uint32_t *>(ws + L.vamax),
                                      static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

// d = 64: the inputs are zero-padded to 128 channels in the workspace (after the d = 128
// call's own region, `inner` bytes), the d = 128 path runs on them, and O's first 64
// channels are copied out.  Zero channels add nothing to S, leave every block maximum (and
// so every scale and code) unchanged, have mean 0 and V scale 0: the result is the d = 64
// definition's.  The kernel's time is set by the softmax per score, not by d.
static sa_status attn_fwd_d64(const void *q, const void *k, const void *v, void *o, int B, int H, int N,
                              float sm_scale, const uint8_t *block_mask, bool causal, cudaStream_t st)
{
    Shape s;
    sa_status r = check_shape(B, H, N, kD, &s);
    if (r != SA_OK) return r;
    size_t inner = align256(ws_layout(s).total);
    if (causal) inner = align256(inner + size_t(s.BH()) * size_t(s.nq()) * size_t(s.nk()));
    const int64_t rows = s.BH() * s.N;
    const size_t tb = align256(size_t(rows) * kD * 2);
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, inner + 4 * tb, &ws)) != SA_OK) return r;
    uint8_t *pq = ws + inner, *pk = pq + tb, *pv = pk + tb, *po = pv + tb;
    if (launch_pad_heads(q, rows, pq, st) != cudaSuccess || launch_pad_heads(k, rows, pk, st) != cudaSuccess ||
        launch_pad_heads(v, rows, pv, st) != cudaSuccess)
        return SA_ERR_CUDA;
    if (causal && block_mask) {
        const size_t attn = align256(ws_layout(s).total);
        if (launch_causal_mask(block_mask, s, ws + attn, st) != cudaSuccess) return SA_ERR_CUDA;
        r = attn_fwd_device(pq, pk, pv, po, s, sm_scale, ws + attn, st, true);
    } else if (causal) {
        r = attn_fwd_device(pq, pk, pv, po, s, sm_scale, nullptr, st, true);
    } else {
        r = attn_fwd_device(pq, pk, pv, po, s, sm_scale, block_mask, st);
    }
    if (r != SA_OK) return r;
    return launch_unpad_heads(po, rows, o, st) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

// A keep mask row of a masked attention call holds at most kMaskedAttnMaxKeyBlocks blocks.
static sa_status check_mask_len(const Shape &s, const void *mask)
{
    return mask && s.nk() > kMaskedAttnMaxKeyBlocks ? SA_ERR_UNSUPPORTED : SA_OK;
}

static sa_status check_d64_call(int B, int H, int N, float sm_scale, std::initializer_list<const void *> ptrs,
                                const void *mask)
{
    Shape s;
    sa_status r = check_shape(B, H, N, kD, &s);
    if (r != SA_OK) return r;
    if ((r = check_mask_len(s, mask)) != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs(ptrs)) != SA_OK) return r;
    return check_device();
}

sa_status sa_attn_fwd(const void *q, const void *k, const void *v, void *o, int B, int H,
                      int N, int d, float sm_scale, const uint8_t *block_mask, void *stream)
{
    if (d == kD / 2) {
        const sa_status r = check_d64_call(B, H, N, sm_scale, {q, k, v, o}, block_mask);
        return r != SA_OK ? r
                          : attn_fwd_d64(q, k, v, o, B, H, N, sm_scale, block_mask, false,
                                         static_cast<cudaStream_t>(stream));
    }
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs({q, k, v, o})) != SA_OK) return r;
    if ((r = check_mask_len(s, block_mask)) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return attn_fwd_device(q, k, v, o, s, sm_scale, block_mask, static_cast<cudaStream_t>(stream));
}

sa_status sa_attn_fwd_host(const void *q, const void *k, const void *v, void *o, int B, int H,
                           int N, int d, float sm_scale, const uint8_t *block_mask, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs({q, k, v, o})) != SA_OK) return r;
    if ((r = check_mask_len(s, block_mask)) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return attn_fwd_host_pipeline(q, k, v, o, s, sm_scale, block_mask, static_cast<cudaStream_t>(stream));
}

sa_status sa_attn_fwd_quantized(const int8_t *q_i8, const float *q_scale, const int8_t *k_i8,
                                const float *k_scale, const uint8_t *v_fp8_t,
                                const float *v_scale, void *o, int B, int H, int N, int d,
                                float sm_scale, const uint8_t *block_mask, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs({q_i8, k_i8, v_fp8_t, o})) != SA_OK) return r;
    if (!q_scale || !k_scale || !v_scale) return SA_ERR_INVALID_ARG;
    if ((r = check_mask_len(s, block_mask)) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return attention_core(q_i8, q_scale, k_i8, k_scale, v_fp8_t, v_scale, o, s, sm_scale,
                          block_mask, static_cast<cudaStream_t>(stream));
}

sa_status sa_block_mask(const void *q, const void *k, int B, int H, int N, int d, int keep_per_row,
                        int keep_diagonal, uint8_t *block_mask, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (keep_per_row < 1) return SA_ERR_INVALID_ARG;
    if (!q || !k || !block_mask) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs({q, k})) != SA_OK) return r;
    if (s.nk() > kMaskMaxKeyBlocks) return SA_ERR_UNSUPPORTED;
    if ((r = check_device()) != SA_OK) return r;
    const size_t qb = align256(size_t(s.BH() * s.nq()) * kD * 4), kb = align256(size_t(s.BH() * s.nk()) * kD * 4);
    const size_t sb = size_t(s.BH() * s.nq()) * size_t(s.nk()) * 8;
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, qb + kb + sb, &ws)) != SA_OK) return r;
    float *qbar = reinterpret_cast<float *>(ws), *kbar = reinterpret_cast<float *>(ws + qb);
    double *scores = reinterpret_cast<double *>(ws + qb + kb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_pool_qk(q, k, s, qbar, kbar, st) != cudaSuccess) return SA_ERR_CUDA;
    return launch_block_select(qbar, kbar, scores, s, keep_per_row, keep_diagonal ? 1 : 0, block_mask, st) == cudaSuccess
               ? SA_OK
               : SA_ERR_CUDA;
}

sa_status sa_debug_pool(const void *q, const void *k, int B, int H, int N, int d, float *qbar,
                        float *kbar, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({q, k, qbar, kbar})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return launch_pool_qk(q, k, s, qbar, kbar, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK
                                                                                              : SA_ERR_CUDA;
}

sa_status sa_w8a8_quantize(const void *x, int rows, int cols, int8_t *codes, float *scales, void *stream)
{
    if (rows < 1 || cols < 1) return SA_ERR_INVALID_ARG;
    if (cols % 8 != 0 || cdiv(rows, 128) > 65535) return SA_ERR_UNSUPPORTED;
    sa_status r = check_ptrs({x, codes, scales});
    if (r != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return launch_w8a8_quantize(x, rows, cols, codes, scales, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SA_OK
               : SA_ERR_CUDA;
}

static sa_status w8a8_gemm_checked(const int8_t *x_codes, const float *x_scales, const int8_t *w_codes,
                                   const float *w_scales, int M, int N, int K, void *y, cudaStream_t st)
{
    const int64_t kpad = cdiv(K, 128) * 128;
    CUtensorMap tx, tw;
    if (!encode_tmap_2d_u8(&tx, x_codes, uint64_t(kpad), uint64_t(M), uint64_t(kpad), 128, kW8a8BoxRows,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d_u8(&tw, w_codes, uint64_t(kpad), uint64_t(N), uint64_t(kpad), 128, kW8a8BoxRows,
                           CU_TENSOR_MAP_SWIZZLE_128B))
        return SA_ERR_CUDA;
    return launch_w8a8_gemm(tx, tw, x_scales, w_scales, M, N, int(kpad / 128), y, st) == cudaSuccess ? SA_OK
                                                                                                : SA_ERR_CUDA;
}

// need_k8: x is quantised here from bf16 rows, read 8 values (16 bytes) at a time
static sa_status check_w8a8_sizes(int M, int N, int K, bool need_k8)
{
    if (M < 1 || N < 1 || K < 1) return SA_ERR_INVALID_ARG;
    if (N % 8 != 0 || (need_k8 && K % 8 != 0)) return SA_ERR_UNSUPPORTED;
    // TMA row coordinates and tile counts are 32-bit; grid rows of the quantiser <= 65535
    if (cdiv(M, 128) > 65535 || cdiv(N, 128) > 65535) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

sa_status sa_w8a8_gemm(const int8_t *x_codes, const float *x_scales, const int8_t *w_codes, const float *w_scales,
                       int M, int N, int K, void *y, void *stream)
{
    sa_status r = check_w8a8_sizes(M, N, K, false);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({x_codes, x_scales, w_codes, w_scales, y})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    return w8a8_gemm_checked(x_codes, x_scales, w_codes, w_scales, M, N, K, y, static_cast<cudaStream_t>(stream));
}

sa_status sa_w8a8_linear(const void *x, const int8_t *w_codes, const float *w_scales, int M, int N, int K,
                         void *y, void *stream)
{
    sa_status r = check_w8a8_sizes(M, N, K, true);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({x, w_codes, w_scales, y})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    const size_t kpad = size_t(cdiv(K, 128)) * 128;
    const size_t cb = align256(size_t(M) * kpad), sb = size_t(cdiv(M, 128)) * size_t(kpad / 128) * 4;
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, cb + sb, &ws)) != SA_OK) return r;
    int8_t *xc = reinterpret_cast<int8_t *>(ws);
    float *xs = reinterpret_cast<float *>(ws + cb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_w8a8_quantize(x, M, K, xc, xs, st) != cudaSuccess) return SA_ERR_CUDA;
    return w8a8_gemm_checked(xc, xs, w_codes, w_scales, M, N, K, y, st);
}

static sa_status check_sla(const Shape &s, int phi, std::initializer_list<const void *> ptrs)
{
    if (phi != 0 && phi != 1) return SA_ERR_INVALID_ARG;
    if (s.nk() > kMaskMaxKeyBlocks) return SA_ERR_UNSUPPORTED;
    return check_ptrs(ptrs);
}

sa_status sa_sla_linear(const void *q, const void *k, const void *v, const uint8_t *classes, int B, int H, int N,
                        int d, int phi, const float *proj, float *out, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!classes) return SA_ERR_INVALID_ARG;
    if ((r = check_sla(s, phi, {q, k, v, out})) != SA_OK) return r;
    if (proj && (r = check_ptrs({proj})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, sla_workspace_bytes(s), &ws)) != SA_OK) return r;
    return launch_sla_linear(q, k, v, classes, s, phi, proj, ws, out, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? SA_OK
               : SA_ERR_CUDA;
}

sa_status sa_sla_fwd(const void *q, const void *k, const void *v, void *o, int B, int H, int N, int d,
                     float sm_scale, const uint8_t *classes, int phi, const float *proj, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale) || !classes) return SA_ERR_INVALID_ARG;
    if ((r = check_sla(s, phi, {q, k, v, o})) != SA_OK) return r;
    if (proj && (r = check_ptrs({proj})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    // workspace: [attention prologue | keep mask | linear-branch states | linear part, fp32]
    const size_t attn = align256(ws_layout(s).total);
    const size_t nmask = size_t(s.BH()) * size_t(s.nq()) * size_t(s.nk());
    const size_t mb = align256(nmask), sb = align256(sla_workspace_bytes(s));
    const size_t lb = size_t(s.BH()) * size_t(s.N) * kD * sizeof(float);
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, attn + mb + sb + lb, &ws)) != SA_OK) return r;
    uint8_t *keep = ws + attn;
    float *lin = reinterpret_cast<float *>(ws + attn + mb + sb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_sla_critical(classes, int64_t(nmask), keep, st) != cudaSuccess) return SA_ERR_CUDA;
    // the linear part first, in fp32; the sparse part's epilogue adds it to O before O's
    // only rounding to bf16
    if (launch_sla_linear(q, k, v, classes, s, phi, proj, ws + attn + mb, lin, st) != cudaSuccess)
        return SA_ERR_CUDA;
    return attn_fwd_device(q, k, v, o, s, sm_scale, keep, st, false, lin);
}

sa_status sa_attn_fwd_causal(const void *q, const void *k, const void *v, void *o, int B, int H, int N, int d,
                             float sm_scale, const uint8_t *block_mask, void *stream)
{
    if (d == kD / 2) {
        const sa_status r = check_d64_call(B, H, N, sm_scale, {q, k, v, o}, block_mask);
        return r != SA_OK ? r
                          : attn_fwd_d64(q, k, v, o, B, H, N, sm_scale, block_mask, true,
                                         static_cast<cudaStream_t>(stream));
    }
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    if ((r = check_ptrs({q, k, v, o})) != SA_OK) return r;
    if ((r = check_mask_len(s, block_mask)) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // without a keep mask the pair kernel runs the causal pattern itself
    if (!block_mask) return attn_fwd_device(q, k, v, o, s, sm_scale, nullptr, st, true);
    // with one: workspace [attention prologue | keep mask intersected with the causal blocks]
    const size_t attn = align256(ws_layout(s).total);
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, attn + size_t(s.BH()) * size_t(s.nq()) * size_t(s.nk()), &ws)) != SA_OK) return r;
    if (launch_causal_mask(block_mask, s, ws + attn, st) != cudaSuccess) return SA_ERR_CUDA;
    return attn_fwd_device(q, k, v, o, s, sm_scale, ws + attn, st, true);
}

sa_status sa_attn_fwd_varlen(const void *q, const void *k, const void *v, void *o, int nseq, const int *seqlens,
                             int H, int d, float sm_scale, int causal, void *stream)
{
    if (nseq < 1 || !seqlens || H < 1) return SA_ERR_INVALID_ARG;
    if (d != kD) return SA_ERR_UNSUPPORTED;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return SA_ERR_INVALID_ARG;
    sa_status r = check_ptrs({q, k, v, o});
    if (r != SA_OK) return r;
    // every sequence is valid on its own; start[i] = its first token in the packed batch
    std::vector<int64_t> start(static_cast<size_t>(nseq) + 1, 0);
    for (int i = 0; i < nseq; ++i) {
        Shape s;
        if ((r = check_shape(1, H, seqlens[i], d, &s)) != SA_OK) return r;
        start[i + 1] = start[i] + seqlens[i];
    }
    if (start[nseq] > INT_MAX / 8 || int64_t(H) * start[nseq] > INT64_MAX / kD) return SA_ERR_INVALID_ARG;
    std::vector<int> ord;
    std::vector<VarlenGroup> groups;
    varlen_groups(nseq, seqlens, H, ord, groups);
    size_t need = 0;
    for (const VarlenGroup &g : groups) {
        Shape s;
        if ((r = check_shape(g.count, H, int(g.nmax), d, &s)) != SA_OK) return r;
        need = std::max(need, align256(ws_layout(s).total));
    }
    // device table after the largest group's workspace: the lengths in group order, then
    // the first row (of d elements) of every head in q, k, v and o
    const size_t lb = align256(size_t(nseq) * sizeof(int)), tb = lb + size_t(nseq) * H * sizeof(int64_t);
    std::vector<uint8_t> table(tb, 0);
    int *lens = reinterpret_cast<int *>(table.data());
    int64_t *rows = reinterpret_cast<int64_t *>(table.data() + lb);
    for (int i = 0; i < nseq; ++i) {
        const int sq = ord[i];
        lens[i] = seqlens[sq];
        for (int h = 0; h < H; ++h) rows[size_t(i) * H + h] = int64_t(H) * start[sq] + int64_t(h) * seqlens[sq];
    }
    if ((r = check_device()) != SA_OK) return r;
    WsLock lock;
    uint8_t *ws = nullptr;
    if ((r = get_workspace(lock, need + tb, &ws)) != SA_OK) return r;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((r = upload_table(table.data(), tb, ws + need, st)) != SA_OK) return r;
    const int *dlens = reinterpret_cast<const int *>(ws + need);
    const int64_t *drows = reinterpret_cast<const int64_t *>(ws + need + lb);
    for (const VarlenGroup &g : groups) {
        Shape s;
        check_shape(g.count, H, int(g.nmax), d, &s);
        SeqTable t;
        t.len = dlens + g.first;
        t.row = drows + size_t(g.first) * H;
        t.H = H;
        if ((r = attn_fwd_device(q, k, v, o, s, sm_scale, nullptr, st, causal != 0, nullptr, t)) != SA_OK) return r;
    }
    return SA_OK;
}

int sa_debug_varlen_groups(int nseq, const int *seqlens, int H, int *group_of)
{
    if (nseq < 1 || !seqlens || !group_of || H < 1) return -1;
    for (int i = 0; i < nseq; ++i)
        if (seqlens[i] < 1) return -1;
    std::vector<int> ord;
    std::vector<VarlenGroup> groups;
    varlen_groups(nseq, seqlens, H, ord, groups);
    for (size_t g = 0; g < groups.size(); ++g)
        for (int i = 0; i < groups[g].count; ++i) group_of[ord[size_t(groups[g].first + i)]] = int(g);
    return int(groups.size());
}

sa_status sa_rope_frequencies(int rot, double base, int scaling, double factor, int original_len,
                              double beta_fast, double beta_slow, double *freqs, float *amplitude)
{
    if (!freqs || !amplitude || rot < 16 || scaling < SA_ROPE_PLAIN || scaling > SA_ROPE_RAMP) return SA_ERR_INVALID_ARG;
    if (rot % 16 != 0 || rot > 256) return SA_ERR_UNSUPPORTED;
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(factor) || factor < 1.0) return SA_ERR_INVALID_ARG;
    const bool ramp = scaling == SA_ROPE_RAMP;
    if (ramp && (original_len < 1 || !std::isfinite(beta_fast) || !(beta_fast > beta_slow) || !(beta_slow > 0.0)))
        return SA_ERR_INVALID_ARG;
    if (scaling == SA_ROPE_BASE) base *= std::pow(factor, double(rot) / (rot - 2));
    // the (real) pair index that turns `turns` times within original_len positions
    auto pair_of = [&](double turns) {
        return rot * std::log(original_len / (turns * 2.0 * 3.14159265358979323846)) / (2.0 * std::log(base));
    };
    double lo = 0.0, hi = 0.0;
    if (ramp) {
        // the borders may lie outside the pairs (a long context turns every pair more than beta_slow
        // times): only the share is clamped
        lo = std::floor(pair_of(beta_fast));
        hi = std::max(std::ceil(pair_of(beta_slow)), lo + 1e-3);  // a step, where both fall on one pair
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        if (scaling == SA_ROPE_LINEAR) {
            freqs[i] = f / factor;
        } else if (ramp) {
            const double share = std::min(1.0, std::max(0.0, (i - lo) / (hi - lo)));  // of the slowed frequency
            freqs[i] = f * (1.0 - share) + f / factor * share;
        } else {
            freqs[i] = f;
        }
    }
    *amplitude = ramp ? float(0.1 * std::log(factor) + 1.0) : 1.0f;
    return SA_OK;
}

sa_status sa_rope(const sa_rope_tensor *tensors, int count, int dtype, int B, int N, int d, int rot,
                  int interleaved, const int32_t *pos, int64_t pos_axis, int64_t pos_batch, int axes,
                  const int *sections, const double *freqs, float amplitude, int inverse, void *stream)
{
    if (!tensors || count < 1 || count > 2 || dtype < SA_BF16 || dtype > SA_FP32) return SA_ERR_INVALID_ARG;
    if (B < 0 || N < 0 || d < 16 || rot < 16 || rot > d || axes < 1) return SA_ERR_INVALID_ARG;
    if (d % 16 != 0 || d > 256 || rot % 16 != 0 || axes > 4) return SA_ERR_UNSUPPORTED;
    if (int64_t(B) * N > (1 << 30)) return SA_ERR_UNSUPPORTED;
    if (!std::isfinite(amplitude) || (!sections && axes != 1)) return SA_ERR_INVALID_ARG;
    RopeArgs a;
    for (int i = 0; i < 3; ++i) a.axis_end[i] = rot / 2;
    if (sections) {
        int sum = 0;
        for (int i = 0; i < axes; ++i) {
            if (sections[i] < 0 || sections[i] > rot / 2) return SA_ERR_INVALID_ARG;
            sum += sections[i];
            if (i < 3) a.axis_end[i] = i < axes - 1 ? sum : rot / 2;
        }
        if (sum != rot / 2) return SA_ERR_INVALID_ARG;
    }
    if (B == 0 || N == 0) return SA_OK;
    const int64_t per16 = dtype == SA_FP32 ? 4 : 8;
    for (int i = 0; i < count; ++i) {
        const sa_rope_tensor &t = tensors[i];
        if (!t.x || !t.y || t.heads < 1) return SA_ERR_INVALID_ARG;
        if (t.heads > 65535) return SA_ERR_UNSUPPORTED;
        if (!aligned16(t.x) || !aligned16(t.y)) return SA_ERR_MISALIGNED;
        for (int64_t st : {t.x_batch, t.x_head, t.x_tok, t.y_batch, t.y_head, t.y_tok})
            if (st % per16 != 0) return SA_ERR_MISALIGNED;
        // an output that is its own copy would be turned several times in place
        if ((B > 1 && t.y_batch == 0) || (t.heads > 1 && t.y_head == 0) || (N > 1 && t.y_tok == 0)) return SA_ERR_INVALID_ARG;
        // in place means element by element: with other strides rows would be written before they are read
        if (t.x == t.y && ((B > 1 && t.x_batch != t.y_batch) || (t.heads > 1 && t.x_head != t.y_head) ||
                           (N > 1 && t.x_tok != t.y_tok)))
            return SA_ERR_INVALID_ARG;
        a.io[i] = RopeIo{t.x, t.y, t.x_batch, t.x_head, t.x_tok, t.y_batch, t.y_head, t.y_tok, t.heads};
    }
    if (count == 2 && (tensors[0].y == tensors[1].y || tensors[0].y == tensors[1].x || tensors[1].y == tensors[0].x))
        return SA_ERR_INVALID_ARG;  // one tensor's blocks would write what the other's read or write
    if (!pos || !freqs) return SA_ERR_INVALID_ARG;
    if (!aligned(pos, 4) || !aligned(freqs, 8)) return SA_ERR_MISALIGNED;
    const sa_status r = check_device();
    if (r != SA_OK) return r;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.inverse = inverse != 0;
    a.pos = pos;
    a.pos_axis_stride = pos_axis;
    a.pos_batch_stride = pos_batch;
    a.freqs = freqs;
    a.amplitude = amplitude;
    return launch_rope(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

static CacheArgs cache_args(int64_t T, const int32_t *tok_start, const int32_t *kv_lens, const int32_t *page_table,
                            int B, int max_pages, const int8_t *k_codes, const float *k_scale, const int8_t *v_codes,
                            const float *v_scale, int num_pages, int H, int d)
{
    CacheArgs a;
    a.k_codes = const_cast<int8_t *>(k_codes);
    a.v_codes = const_cast<int8_t *>(v_codes);
    a.k_scale = const_cast<float *>(k_scale);
    a.v_scale = const_cast<float *>(v_scale);
    a.tok_start = tok_start;
    a.kv_lens = kv_lens;
    a.table = page_table;
    a.T = int(T);
    a.B = B;
    a.H = H;
    a.d = d;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    return a;
}

sa_status sa_cache_append(const void *k, const void *v, int dtype, int64_t T, int64_t k_tok, int64_t v_tok,
                          const int32_t *tok_start, const int32_t *kv_lens, const int32_t *page_table, int B,
                          int max_pages, int8_t *k_codes, float *k_scale, int8_t *v_codes, float *v_scale,
                          int num_pages, int H, int d, void *stream)
{
    if (dtype != SA_BF16 && dtype != SA_FP16) return SA_ERR_INVALID_ARG;
    sa_status r = check_cache(T, B, H, d, max_pages, num_pages, tok_start, kv_lens, page_table, k_codes, k_scale,
                              v_codes, v_scale);
    if (r != SA_OK || T == 0) return r;
    if ((r = check_tokens(k, k_tok, int64_t(H) * d)) != SA_OK) return r;
    if ((r = check_tokens(v, v_tok, int64_t(H) * d)) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    CacheArgs a = cache_args(T, tok_start, kv_lens, page_table, B, max_pages, k_codes, k_scale, v_codes, v_scale,
                             num_pages, H, d);
    a.k = k;
    a.v = v;
    a.k_stride = k_tok;
    a.v_stride = v_tok;
    return launch_cache_append(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_cache_read(void *k, void *v, int dtype, int64_t T, const int32_t *tok_start,
                        const int32_t *kv_lens, const int32_t *page_table, int B, int max_pages,
                        const int8_t *k_codes, const float *k_scale, const int8_t *v_codes,
                        const float *v_scale, int num_pages, int H, int d, void *stream)
{
    if (dtype < SA_BF16 || dtype > SA_FP32) return SA_ERR_INVALID_ARG;
    sa_status r = check_cache(T, B, H, d, max_pages, num_pages, tok_start, kv_lens, page_table, k_codes, k_scale,
                              v_codes, v_scale);
    if (r != SA_OK || T == 0) return r;
    if (!k && !v) return SA_ERR_INVALID_ARG;
    if ((k && !aligned16(k)) || (v && !aligned16(v))) return SA_ERR_MISALIGNED;
    if ((r = check_device()) != SA_OK) return r;
    CacheArgs a = cache_args(T, tok_start, kv_lens, page_table, B, max_pages, k_codes, k_scale, v_codes, v_scale,
                             num_pages, H, d);
    a.k = k;
    a.v = v;
    return launch_cache_read(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

static std::atomic<int> g_cache_attn_quit{-1};

void sa_debug_cache_attn_quit(int worker) { g_cache_attn_quit.store(worker, std::memory_order_relaxed); }

// The query side of an attention call over the cache.
static sa_status check_group(int64_t T, int H, int group)
{
    if (group < 1) return SA_ERR_INVALID_ARG;
    if (int64_t(H) * group > 65535 || T * group > (1 << 30) || T * H * group > (int64_t(1) << 34))
        return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

sa_status sa_cache_attn(const void *q, void *o, float *lse, int dtype, int64_t T, int64_t q_tok,
                        const int32_t *tok_start, const int32_t *kv_lens, const int32_t *page_table, int B,
                        int max_pages, const int8_t *k_codes, const float *k_scale, const int8_t *v_codes,
                        const float *v_scale, int num_pages, int H, int group, int d, int causal, int window,
                        float sm_scale, void *workspace, size_t workspace_bytes, void *stream)
{
    if ((dtype != SA_BF16 && dtype != SA_FP16) || window < 0 || !std::isfinite(sm_scale) || sm_scale <= 0.0f)
        return SA_ERR_INVALID_ARG;
    sa_status r = check_cache(T, B, H, d, max_pages, num_pages, tok_start, kv_lens, page_table, k_codes, k_scale,
                              v_codes, v_scale);
    if (r == SA_OK) r = check_group(T, H, group);
    if (r != SA_OK || T == 0) return r;
    if ((r = check_tokens(q, q_tok, int64_t(H) * group * d)) != SA_OK) return r;
    if (!o || !workspace) return SA_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(workspace) || !aligned(lse, 4)) return SA_ERR_MISALIGNED;
    // blocks that share a query row write it while others may still read it
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
    const int64_t width = int64_t(H) * group * d;
    if (o0 < q0 + 2 * uint64_t((T - 1) * q_tok + width) && q0 < o0 + 2 * uint64_t(T * width)) return SA_ERR_INVALID_ARG;
    if ((r = check_device()) != SA_OK) return r;
    if (workspace_bytes < sa_cache_attn_workspace_bytes(T, B, H, group, d)) return SA_ERR_INVALID_ARG;
    CUtensorMap tm_k, tm_v;
    const uint64_t lines = uint64_t(num_pages) * uint64_t(H) * uint64_t(d) / 2;  // of 128 bytes
    if (!encode_tmap_2d_u8(&tm_k, k_codes, 128, lines, 128, 128, uint32_t(d / 2), CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d_u8(&tm_v, v_codes, 128, lines, 128, 128, uint32_t(d / 2), CU_TENSOR_MAP_SWIZZLE_128B))
        return SA_ERR_CUDA;
    CacheAttnArgs a;
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.dtype = dtype;
    a.q_stride = q_tok;
    a.k_codes = k_codes;
    a.v_codes = v_codes;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.tok_start = tok_start;
    a.kv_lens = kv_lens;
    a.table = page_table;
    a.T = int(T);
    a.B = B;
    a.H = H;
    a.G = group;
    a.d = d;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.causal = causal != 0;
    a.window = std::min(window, 1 << 30);
    a.sm_scale = sm_scale;
    a.quit = g_cache_attn_quit.load(std::memory_order_relaxed);
    return launch_cache_attn(tm_k, tm_v, a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK
                                                                                                       : SA_ERR_CUDA;
}

size_t sa_cache_attn_workspace_bytes(int64_t T, int B, int H, int group, int d)
{
    if (check_cache_sizes(T, B, H, d) != SA_OK || check_group(T, H, group) != SA_OK) return 0;
    const int sms = device_sms();
    return sms < 1 ? 0 : cache_attn_workspace(sms, T, B, group, d);
}

int64_t sa_debug_cache_steps(int n, int len, int group, int causal, int window)
{
    if (n < 0 || len < 0 || len > (1 << 30) || group < 1 || int64_t(n) * group > (1 << 30) || window < 0) return -1;
    return steps_of(n, len, group, causal, std::min(window, 1 << 30), 0, 1);
}

sa_status sa_debug_qk_s32(const int8_t *q_i8, const int8_t *k_i8, int B, int H, int N, int d,
                          int32_t *s_out, void *stream)
{
    Shape s;
    sa_status r = check_shape(B, H, N, d, &s);
    if (r != SA_OK) return r;
    if ((r = check_ptrs({q_i8, k_i8, s_out})) != SA_OK) return r;
    if ((r = check_device()) != SA_OK) return r;
    CUtensorMap tq, tk;
    const uint64_t rows = uint64_t(s.BH() * s.Npad());
    if (!encode_tmap_2d_u8(&tq, q_i8, kD, rows, kD, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d_u8(&tk, k_i8, kD, rows, kD, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return SA_ERR_CUDA;
    return launch_debug_qk_s32(tq, tk, int(s.BH()), int(s.Npad()), s_out,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SA_OK
               : SA_ERR_CUDA;
}

sa_status sa_debug_wait_timeout(int timeout_us, void *stream)
{
    if (timeout_us < 1 || timeout_us > 10000000) return SA_ERR_INVALID_ARG;
    sa_status r = check_device();
    if (r != SA_OK) return r;
    return launch_debug_wait_timeout(timeout_us, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SA_OK
               : SA_ERR_CUDA;
}

sa_status sa_debug_mma_peak(int kind, int reps, void *stream)
{
    if ((kind != 0 && kind != 1) || reps < 1 || reps > (1 << 20)) return SA_ERR_INVALID_ARG;
    sa_status r = check_device();
    if (r != SA_OK) return r;
    return launch_mma_peak(kind, reps, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_get_device_status(void)
{
    int st = 0, st_w8a8 = 0, st_peak = 0, st_sla = 0, st_cache = 0, st_cattn = 0, st_chunk = 0;
    if (read_and_clear_cache_status(&st_cache) != cudaSuccess || read_and_clear_cache_attn_status(&st_cattn) != cudaSuccess ||
        read_and_clear_cache_chunk_status(&st_chunk) != cudaSuccess ||
        read_and_clear_status(&st) != cudaSuccess || read_and_clear_w8a8_status(&st_w8a8) != cudaSuccess ||
        read_and_clear_peak_status(&st_peak) != cudaSuccess || read_and_clear_sla_status(&st_sla) != cudaSuccess)
        return SA_ERR_CUDA;
    if (st != 0 || st_w8a8 != 0 || st_peak != 0 || st_sla != 0 || st_cattn == SA_ERR_DEVICE_TIMEOUT ||
        st_chunk == SA_ERR_DEVICE_TIMEOUT)
        return SA_ERR_DEVICE_TIMEOUT;
    return st_cache == 0 && st_cattn == 0 && st_chunk == 0 ? SA_OK : SA_ERR_BAD_INDEX;
}

const char *sa_status_string(sa_status s)
{
    switch (s) {
    case SA_OK: return "SA_OK";
    case SA_ERR_INVALID_ARG: return "SA_ERR_INVALID_ARG";
    case SA_ERR_UNSUPPORTED: return "SA_ERR_UNSUPPORTED";
    case SA_ERR_MISALIGNED: return "SA_ERR_MISALIGNED";
    case SA_ERR_CUDA: return "SA_ERR_CUDA";
    case SA_ERR_OOM: return "SA_ERR_OOM";
    case SA_ERR_DEVICE_TIMEOUT: return "SA_ERR_DEVICE_TIMEOUT";
    case SA_ERR_SCRATCH_LIMIT: return "SA_ERR_SCRATCH_LIMIT";
    case SA_ERR_BAD_INDEX: return "SA_ERR_BAD_INDEX";
    }
    return "SA_ERR_UNKNOWN";
}

size_t sa_workspace_bytes(int B, int H, int N, int d)
{
    Shape s;
    if (check_shape(B, H, N, d == kD / 2 ? kD : d, &s) != SA_OK) return 0;
    if (d != kD / 2) return ws_layout(s).total;
    // d = 64: the d = 128 workspace, then the four zero-padded copies of q, k, v and o
    return align256(ws_layout(s).total) + 4 * align256(size_t(s.BH()) * size_t(s.N) * kD * 2);
}

sa_status sa_release_workspace(void)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SA_ERR_CUDA;
    WsLock lock(g_ws_mutex);
    DeviceWs &w = g_ws[dev];
    if (w.ptr) {
        if (cudaDeviceSynchronize() != cudaSuccess) return SA_ERR_CUDA;
        cudaFree(w.ptr);
        w.ptr = nullptr;
        w.bytes = 0;
    }
    HostStage &h = g_stage[dev];
    if (h.ptr) {
        if (cudaEventSynchronize(h.ev) != cudaSuccess) return SA_ERR_CUDA;
        cudaFreeHost(h.ptr);
        h.ptr = nullptr;
        h.bytes = 0;
    }
    return SA_OK;
}

int64_t sa_padded_len(int N) { return N < 1 ? 0 : sa::padded_len(N); }

}  // extern "C"
