"""The rotary and cache entry points without a GPU: bad arguments are refused on the host
before any CUDA call, and the rotation frequencies follow their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

FAKE = 1 << 20       # 16-byte aligned, never dereferenced
ODD = FAKE + 8       # aligned to 8 only
SCALE = ctypes.c_float(0.088)


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=0, T=8, ks=1024, vs=1024, starts=FAKE, lens=FAKE, table=FAKE, B=2, max_pages=4,
             kc=FAKE, kscale=FAKE, vc=FAKE, vscale=FAKE, pages=16, H=8, d=128)
    a.update(kw)
    return lib.sa_cache_append(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), 1), (dict(starts=None), 1), (dict(vscale=None), 1), (dict(dtype=2), 1), (dict(T=-1), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(ks=1016), 1),
    (dict(d=96), 2), (dict(T=(1 << 30) + 1), 2), (dict(H=65536, ks=1 << 24, vs=1 << 24), 2),
    (dict(max_pages=(1 << 24) + 1), 2), (dict(pages=1 << 25), 2), (dict(B=(1 << 20) + 1), 2),
    (dict(k=ODD), 3), (dict(kc=ODD), 3), (dict(vs=1028), 3), (dict(lens=FAKE + 2), 3), (dict(kscale=FAKE + 1), 3),
    (dict(T=0, k=None, kc=None), 0),
])
def test_append_refusals(libsa, kw, expect):
    assert _append(libsa.raw_library(), **kw) == expect


def _read(lib, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=2, T=8, starts=FAKE, lens=FAKE, table=FAKE, B=2, max_pages=4, kc=FAKE, kscale=FAKE,
             vc=FAKE, vscale=FAKE, pages=16, H=8, d=128)
    a.update(kw)
    return lib.sa_cache_read(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None, v=None), 1), (dict(dtype=3), 1), (dict(table=None), 1), (dict(d=32), 2), (dict(v=ODD), 3),
    (dict(k=None, v=ODD), 3), (dict(T=0, k=None, v=None), 0),
])
def test_read_refusals(libsa, kw, expect):
    assert _read(libsa.raw_library(), **kw) == expect


def _attn(lib, **kw):
    a = dict(q=FAKE, o=FAKE + (1 << 24), lse=None, dtype=0, T=8, qs=2048, starts=FAKE, lens=FAKE, table=FAKE, B=2, max_pages=4,
             kc=FAKE, kscale=FAKE, vc=FAKE, vscale=FAKE, pages=16, H=8, group=2, d=128, causal=1, window=0, scale=SCALE,
             ws=FAKE, nbytes=1 << 40)
    a.update(kw)
    return lib.sa_cache_attn(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(dtype=2), 1), (dict(group=0), 1), (dict(window=-1), 1),
    (dict(scale=ctypes.c_float(0.0)), 1), (dict(scale=ctypes.c_float(math.nan)), 1), (dict(scale=ctypes.c_float(math.inf)), 1),
    (dict(qs=2040), 1), (dict(d=80), 2), (dict(group=8192), 2), (dict(T=1 << 30), 2), (dict(o=ODD), 3), (dict(ws=ODD), 3), (dict(o=FAKE), 1),
    (dict(lse=FAKE + 2), 3), (dict(qs=2052), 3), (dict(T=0, q=None, o=None, ws=None), 0),
])
def test_attn_refusals(libsa, kw, expect):
    assert _attn(libsa.raw_library(), **kw) == expect


def test_attn_refuses_an_output_over_its_queries(libsa):
    """T tokens of H * group * d = 2048 values with a stride of 4096: outputs that reach the first
    or the last 16 bytes of the span of q."""
    lib, T = libsa.raw_library(), 8
    span, size = 2 * ((T - 1) * 4096 + 2048), 2 * T * 2048
    for o in (FAKE - size + 16, FAKE, FAKE + span - 16):
        assert _attn(lib, q=FAKE, o=o, qs=4096) == 1


def test_attn_workspace_of_refused_sizes_is_zero(libsa):
    f = libsa.raw_library().sa_cache_attn_workspace_bytes
    assert f(1, 0, 8, 1, 128) == 0 and f(1, 1, 8, 1, 96) == 0 and f(1, 1, 8, 0, 128) == 0 and f(-1, 1, 8, 1, 128) == 0


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("x_batch", "x_head", "x_tok", "y_batch", "y_head", "y_tok")] + [("heads", ctypes.c_int)]


def _rope(lib, **kw):
    a = dict(count=1, dtype=0, B=1, N=8, d=128, rot=128, inter=0, pos=FAKE, pa=0, pb=0, axes=1, sections=None, freqs=FAKE,
             amp=ctypes.c_float(1.0), inverse=0)
    t = dict(x=FAKE, y=FAKE, x_batch=0, x_head=1024, x_tok=128, y_batch=0, y_head=1024, y_tok=128, heads=4)
    t.update({k: kw.pop(k) for k in list(kw) if k in t})
    a.update(kw)
    arr = (RopeTensor * 2)(RopeTensor(**t), RopeTensor(**t))
    return lib.sa_rope(arr, *a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(count=0), 1), (dict(count=3), 1), (dict(dtype=3), 1), (dict(N=-1), 1), (dict(rot=144), 1), (dict(rot=0), 1),
    (dict(x=None), 1), (dict(heads=0), 1), (dict(pos=None), 1), (dict(freqs=None), 1), (dict(axes=2), 1),
    (dict(axes=3, sections=(ctypes.c_int * 3)(22, 21, 20)), 1), (dict(axes=2, sections=(ctypes.c_int * 2)(-1, 65)), 1),
    (dict(amp=ctypes.c_float(math.inf)), 1), (dict(d=120, rot=16), 2), (dict(d=272, rot=16), 2), (dict(rot=24), 2),
    (dict(axes=5, sections=(ctypes.c_int * 5)(64, 0, 0, 0, 0)), 2), (dict(B=1 << 20, N=1 << 20), 2), (dict(y=ODD), 3),
    (dict(x_tok=132), 3), (dict(freqs=FAKE + 4), 3), (dict(pos=FAKE + 2), 3), (dict(N=0, x=None), 0), (dict(B=0), 0),
])
def test_rope_refusals(libsa, kw, expect):
    assert _rope(libsa.raw_library(), **kw) == expect


@pytest.mark.parametrize("kw", [dict(y_head=0), dict(y_tok=0), dict(B=2)])
def test_rope_refuses_an_output_over_itself(libsa, kw):
    # such an output would be read again after it was turned; broadcast inputs and sizes of one are fine
    assert _rope(libsa.raw_library(), **kw) == 1
    assert _rope(libsa.raw_library(), x_head=0, x_tok=0, y_head=0, y_tok=0, B=0) == 0


@pytest.mark.parametrize("kw", [dict(y_head=1152), dict(y_tok=256), dict(x_tok=0), dict(x_head=0), dict(B=2, y_batch=1 << 16)])
def test_rope_refuses_in_place_with_other_strides(libsa, kw):
    assert _rope(libsa.raw_library(), **kw) == 1


def test_rope_refuses_tensors_that_write_each_other(libsa):
    lib = libsa.raw_library()

    def call(x0, y0, x1, y1):
        t = (RopeTensor * 2)(*(RopeTensor(x, y, 0, 1024, 128, 0, 1024, 128, 4) for x, y in ((x0, y0), (x1, y1))))
        # a call that passes this check is refused for its misaligned positions
        return lib.sa_rope(t, 2, 0, 1, 8, 128, 128, 0, FAKE + 2, 0, 0, 1, None, FAKE, ctypes.c_float(1.0), 0, None)

    a, b, c = FAKE, FAKE + (1 << 20), FAKE + (2 << 20)
    assert call(a, b, c, b) == 1    # one output for both
    assert call(a, b, b, c) == 1    # q' over k
    assert call(a, c, b, a) == 1    # k' over q
    assert call(a, a, b, b) == 3    # in place, each its own
    assert call(a, b, a, c) == 3    # one input for both


def test_binding_refusals(libsa):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = tuple(libsa.sa_cache_alloc(4, 2, 128, device="cpu"))
    i32 = dict(dtype=torch.int32)
    seqs = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 4, **i32)
    with pytest.raises(ValueError):
        libsa.sa_cache_append(cache, x, x, *seqs)                        # CPU tensors
    with pytest.raises(ValueError):
        libsa.sa_cache_read(cache, 4, *seqs)
    with pytest.raises(ValueError):
        libsa.sa_cache_attn(cache, x, *seqs)
    with pytest.raises(ValueError):
        libsa.sa_cache_attn(cache, torch.zeros(4, 3, 128), *seqs)        # 3 heads over 2
    with pytest.raises(ValueError):
        libsa.sa_cache_attn(cache[:2] + (cache[2][:3], cache[3]), x, *seqs)
    with pytest.raises(ValueError):
        libsa.sa_cache_attn(cache, x, seqs[0][:1], *seqs[1:])            # tok_start without its end
    with pytest.raises(ValueError):
        libsa.sa_rope(x, None, seqs[1], torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        libsa.sa_rope_frequencies(128, scaling="other", device="cpu")


@pytest.mark.parametrize("kw,status", [
    (dict(rot=24), 2), (dict(rot=0), 1), (dict(rot=272), 2), (dict(rot=64, base=1.0), 1), (dict(rot=64, factor=0.5), 1),
    (dict(rot=64, base=math.nan), 1), (dict(rot=64, scaling="ramp"), 1),
    (dict(rot=64, scaling="ramp", original_len=4096, beta_fast=1.0, beta_slow=1.0), 1),
])
def test_frequencies_refusals(libsa, kw, status):
    with pytest.raises(libsa.SAError) as e:
        libsa.sa_rope_frequencies(device="cpu", **kw)
    assert e.value.status == status


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 10000.0), (96, 500000.0)])
def test_frequencies_follow_their_formulas(libsa, rot, base):
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    f, a = libsa.sa_rope_frequencies(rot, base, device="cpu")
    assert np.allclose(f.numpy(), plain, rtol=1e-14, atol=0) and a == 1.0
    f, a = libsa.sa_rope_frequencies(rot, base, "linear", 8.0, device="cpu")
    assert np.allclose(f.numpy(), plain / 8.0, rtol=1e-14, atol=0) and a == 1.0
    f, _ = libsa.sa_rope_frequencies(rot, base, "base", 8.0, device="cpu")
    assert f[0] == 1.0 and math.isclose(f[-1].item(), plain[-1] / 8.0, rel_tol=1e-12)
    L, factor, fast, slow = 4096, 8.0, 32.0, 1.0
    f, a = libsa.sa_rope_frequencies(rot, base, "ramp", factor, L, fast, slow, device="cpu")
    turns = L * plain / (2 * math.pi)
    share = (plain - f.numpy()) / (plain - plain / factor)
    assert np.all(np.abs(share[turns >= fast * base ** (2 / rot)]) < 1e-12)      # a pair beyond the border
    assert np.all(np.abs(share[turns <= slow / base ** (2 / rot)] - 1) < 1e-12)
    assert np.all(np.diff(share) >= -1e-12) and math.isclose(a, 0.1 * math.log(factor) + 1, rel_tol=1e-6)
    f, a = libsa.sa_rope_frequencies(rot, base, "ramp", 1.0, L, fast, slow, device="cpu")
    assert np.allclose(f.numpy(), plain, rtol=1e-14, atol=0) and a == 1.0
