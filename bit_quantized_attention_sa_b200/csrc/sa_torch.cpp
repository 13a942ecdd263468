// sa_torch.cpp -- the torch side of the serving calls (sa_rope, sa_cache_append, sa_cache_read,
// sa_cache_attn): checks of the tensors, outputs and workspaces from torch's allocator, the
// current stream, and the call of the C ABI in include/sa.h.  Nothing is computed here.
//
// A decoding step makes several such calls for every layer, each of a few microseconds on the
// GPU; the same checks in Python took 20 to 30 us a call, so they are made here (5 to 11 us).
#include <climits>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include "../../include/sa.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using std::optional;

[[noreturn]] void refuse(const char *why) { throw py::value_error(why); }

py::object *g_error = nullptr;  // binding.SAError

void done(sa_status status, const char *what)
{
    if (status == SA_OK) return;
    PyErr_SetObject(g_error->ptr(), (*g_error)(int(status), what).ptr());
    throw py::error_already_set();
}

int dtype_of(const Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kBFloat16: return SA_BF16;
    case at::kHalf: return SA_FP16;
    case at::kFloat: return SA_FP32;
    default: return -1;
    }
}

int cuda_index(const Tensor &t) { return t.is_cuda() ? int(t.get_device()) : -1; }

void *stream_of(int index) { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream(); }

int as_int(int64_t n, const char *why)
{
    if (n < INT_MIN || n > INT_MAX) refuse(why);
    return int(n);
}

// ---- rotary positions

struct View {
    int64_t B, N, H, batch, head, tok;
};

// [B, H, N, d], or packed [T, H, d]; the stride of a dimension of one is any number, and not used.
View view_of(const Tensor &t)
{
    const auto n = t.sizes(), s = t.strides();
    if (t.dim() == 4)
        return {n[0], n[2], n[1], n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, n[2] > 1 ? s[2] : 0};
    return {1, n[0], n[1], 0, n[1] > 1 ? s[1] : 0, n[0] > 1 ? s[0] : 0};
}

View describe(sa_rope_tensor &d, const Tensor &x, const Tensor &y, const Tensor &like, int index)
{
    if (cuda_index(x) != index || x.scalar_type() != like.scalar_type() || x.dim() != like.dim() ||
        x.size(-1) != like.size(-1))
        refuse("q and k differ in dtype, device, layout or head size");
    if (cuda_index(y) != index || y.scalar_type() != x.scalar_type() || y.sizes() != x.sizes())
        refuse("out must have q's and k's dtypes, devices and shapes");
    if (x.stride(-1) != 1 || y.stride(-1) != 1) refuse("q, k and out must have contiguous channels");
    const View a = view_of(x), b = view_of(y);
    d = {x.data_ptr(), y.data_ptr(), a.batch, a.head, a.tok, b.batch, b.head, b.tok, as_int(a.H, "too many heads")};
    return a;
}

py::object rope(const Tensor &q, const optional<Tensor> &k, const Tensor &pos, const Tensor &freqs, optional<int64_t> rot_,
                bool interleaved, const optional<std::vector<int64_t>> &sections, double amplitude, bool inverse,
                const optional<Tensor> &out_q, const optional<Tensor> &out_k)
{
    const int index = cuda_index(q), dtype = dtype_of(q);
    if (index < 0 || dtype < 0 || (q.dim() != 3 && q.dim() != 4))
        refuse("q and k must be bf16, fp16 or fp32 CUDA tensors [B, H, N, d] or [T, H, d]");
    const c10::cuda::CUDAGuard guard{c10::DeviceIndex(index)};
    const Tensor yq = out_q ? *out_q : at::empty(q.sizes(), q.options());
    Tensor yk;
    if (k) yk = out_k ? *out_k : at::empty(k->sizes(), k->options());
    sa_rope_tensor io[2];
    const View a = describe(io[0], q, yq, q, index);
    if (k) {
        const View b = describe(io[1], *k, yk, q, index);
        if (b.B != a.B || b.N != a.N) refuse("q and k have different tokens");
    }
    const int64_t d = q.size(-1), rot = rot_.value_or(d);
    int axes = 1, counts[8];
    if (sections) {
        if (sections->empty() || sections->size() > 8) refuse("sections must be the pair counts of 1 to 4 axes");
        axes = int(sections->size());
        for (int i = 0; i < axes; ++i) counts[i] = as_int((*sections)[size_t(i)], "a section is too large");
    }
    const int64_t lead = sections ? 1 : 0, dims = pos.dim() - lead;
    if (pos.scalar_type() != at::kInt || cuda_index(pos) != index || !pos.is_contiguous() || (dims != 1 && dims != 2) ||
        (lead && pos.size(0) != axes) || pos.size(-1) != a.N || (dims == 2 && pos.size(lead) != a.B))
        refuse("pos must be contiguous int32 [N], [B, N] or [T] on q's device, after one row for each section");
    if (freqs.scalar_type() != at::kDouble || cuda_index(freqs) != index || !freqs.is_contiguous() ||
        freqs.numel() != rot / 2)
        refuse("freqs must be a contiguous fp64 tensor of rot / 2 values on q's device");
    done(sa_rope(io, k ? 2 : 1, dtype, as_int(a.B, "too many batches"), as_int(a.N, "too many tokens"),
                 as_int(d, "d is too large"), as_int(rot, "rot is too large"), interleaved,
                 static_cast<const int32_t *>(pos.data_ptr()), dims == 2 ? a.N * a.B : a.N, dims == 2 ? a.N : 0, axes,
                 sections ? counts : nullptr, static_cast<const double *>(freqs.data_ptr()), float(amplitude), inverse,
                 stream_of(index)),
         "sa_rope");
    if (!k) return py::cast(yq);
    return py::make_tuple(yq, yk);
}

// ---- the cache

struct Cache {
    const Tensor &kc, &ks, &vc, &vs;
    const int32_t *starts, *lens, *table;
    int B, max_pages, pages, H, d;
    int8_t *k_codes() const { return static_cast<int8_t *>(kc.data_ptr()); }
    int8_t *v_codes() const { return static_cast<int8_t *>(vc.data_ptr()); }
    float *k_scale() const { return static_cast<float *>(ks.data_ptr()); }
    float *v_scale() const { return static_cast<float *>(vs.data_ptr()); }
};

Cache cache_of(const Tensor &kc, const Tensor &ks, const Tensor &vc, const Tensor &vs, const Tensor &starts,
               const Tensor &lens, const Tensor &table, int index)
{
    if (kc.dim() != 4 || kc.size(2) != SA_CACHE_PAGE || kc.scalar_type() != at::kChar || vc.scalar_type() != at::kChar ||
        vc.sizes() != kc.sizes())
        refuse("the cache's codes must be int8 [pages, heads, 64, d]");
    for (const Tensor *s : {&ks, &vs})
        if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != kc.size(0) || s->size(1) != kc.size(1))
            refuse("the cache's scales must be fp32 [pages, heads]");
    const int64_t B = lens.dim() == 1 ? lens.size(0) : -1;
    if (starts.scalar_type() != at::kInt || lens.scalar_type() != at::kInt || table.scalar_type() != at::kInt ||
        starts.dim() != 1 || starts.size(0) != B + 1 || table.dim() != 2 || table.size(0) != B)
        refuse("tok_start, kv_lens and page_table must be int32 [B + 1], [B] and [B, max_pages]");
    for (const Tensor *t : {&kc, &ks, &vc, &vs, &starts, &lens, &table})
        if (index < 0 || cuda_index(*t) != index || !t->is_contiguous())
            refuse("the cache and the sequences' arrays must be contiguous, on the tokens' CUDA device");
    const char *large = "a size of the cache is too large";
    return {kc, ks, vc, vs, static_cast<const int32_t *>(starts.data_ptr()), static_cast<const int32_t *>(lens.data_ptr()),
            static_cast<const int32_t *>(table.data_ptr()), as_int(B, large), as_int(table.size(1), large),
            as_int(kc.size(0), large), as_int(kc.size(1), large), as_int(kc.size(3), large)};
}

// Packed tokens [T, heads, d], strided over tokens only; returns the token stride.
int64_t tokens_of(const Tensor &t, int index, int d, const char *why)
{
    if (cuda_index(t) != index || t.dim() != 3 || (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf) ||
        t.size(2) != d || t.size(1) < 1)
        refuse(why);
    if (t.size(0) > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != d))) refuse(why);
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * d;
}

void append(const Tensor &kc, const Tensor &ks, const Tensor &vc, const Tensor &vs, const Tensor &k, const Tensor &v,
            const Tensor &starts, const Tensor &lens, const Tensor &table)
{
    const int index = cuda_index(k);
    const Cache c = cache_of(kc, ks, vc, vs, starts, lens, table, index);
    const char *why = "k and v must be bf16 or fp16 CUDA tensors [T, heads, d] with the cache's heads, one after another";
    const int64_t k_tok = tokens_of(k, index, c.d, why), v_tok = tokens_of(v, index, c.d, why);
    if (k.size(1) != c.H || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type()) refuse(why);
    const c10::cuda::CUDAGuard guard{c10::DeviceIndex(index)};
    done(sa_cache_append(k.data_ptr(), v.data_ptr(), dtype_of(k), k.size(0), k_tok, v_tok, c.starts, c.lens, c.table, c.B,
                         c.max_pages, c.k_codes(), c.k_scale(), c.v_codes(), c.v_scale(), c.pages, c.H, c.d,
                         stream_of(index)),
         "sa_cache_append");
}

py::object read_tokens(const Tensor &kc, const Tensor &ks, const Tensor &vc, const Tensor &vs, int64_t tokens,
                const Tensor &starts, const Tensor &lens, const Tensor &table, const py::object &dtype)
{
    const int index = cuda_index(kc);
    const Cache c = cache_of(kc, ks, vc, vs, starts, lens, table, index);
    if (tokens < 0 || !THPDtype_Check(dtype.ptr())) refuse("tokens must not be negative, dtype be a torch dtype");
    const c10::cuda::CUDAGuard guard{c10::DeviceIndex(index)};
    const auto options = ks.options().dtype(reinterpret_cast<THPDtype *>(dtype.ptr())->scalar_type);
    const Tensor k = at::empty({tokens, c.H, c.d}, options), v = at::empty({tokens, c.H, c.d}, options);
    if (dtype_of(k) < 0) refuse("dtype must be bf16, fp16 or fp32");
    done(sa_cache_read(k.data_ptr(), v.data_ptr(), dtype_of(k), tokens, c.starts, c.lens, c.table, c.B, c.max_pages,
                       c.k_codes(), c.k_scale(), c.v_codes(), c.v_scale(), c.pages, c.H, c.d, stream_of(index)),
         "sa_cache_read");
    return py::make_tuple(k, v);
}

py::object attn(const Tensor &kc, const Tensor &ks, const Tensor &vc, const Tensor &vs, const Tensor &q,
                const Tensor &starts, const Tensor &lens, const Tensor &table, bool causal, int64_t window,
                optional<double> sm_scale, bool return_lse, const optional<Tensor> &out)
{
    const int index = cuda_index(q);
    const Cache c = cache_of(kc, ks, vc, vs, starts, lens, table, index);
    const char *why = "q must be a bf16 or fp16 CUDA tensor [T, query heads, d], the heads one after another and a "
                      "multiple of the cache's";
    const int64_t q_tok = tokens_of(q, index, c.d, why), T = q.size(0);
    if (c.H < 1 || q.size(1) % c.H != 0) refuse(why);
    const int group = as_int(q.size(1) / c.H, why);
    if (out && (out->scalar_type() != q.scalar_type() || cuda_index(*out) != index || out->sizes() != q.sizes() ||
                !out->is_contiguous()))
        refuse("out must be a contiguous tensor of q's dtype, device and shape");
    const c10::cuda::CUDAGuard guard{c10::DeviceIndex(index)};
    const Tensor o = out ? *out : at::empty(q.sizes(), q.options());
    Tensor lse;
    if (return_lse) lse = at::empty({T, q.size(1)}, ks.options());
    // the workspace is torch's, so that calls on several streams and captured graphs have their own
    const size_t need = sa_cache_attn_workspace_bytes(T, c.B, c.H, group, c.d);
    const Tensor ws = at::empty({int64_t(need)}, kc.options());
    done(sa_cache_attn(q.data_ptr(), o.data_ptr(), return_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, dtype_of(q),
                       T, q_tok, c.starts, c.lens, c.table, c.B, c.max_pages, c.k_codes(), c.k_scale(), c.v_codes(),
                       c.v_scale(), c.pages, c.H, group, c.d, causal, int(std::min<int64_t>(std::max<int64_t>(window, -1), 1 << 30)),
                       sm_scale ? float(*sm_scale) : float(1.0 / std::sqrt(double(c.d))), ws.data_ptr(), need,
                       stream_of(index)),
         "sa_cache_attn");
    if (!return_lse) return py::cast(o);
    return py::make_tuple(o, lse);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    m.def("set_error", [](py::object cls) { g_error = new py::object(std::move(cls)); });
    m.def("rope", &rope);
    m.def("append", &append);
    m.def("read", &read_tokens);
    m.def("attn", &attn);
}
