"""Rotary positions on the GPU against the 64-bit formula: layouts, parts of the head, axes,
types, strides, in place, far positions, and the transposed map."""
import pytest
import torch

from _cache_ref import HALF_STEP, rope_ref

pytestmark = pytest.mark.gpu


def _check(y, x, pos, freqs, rot, **kw):
    """Half a step of the output type; the sine, cosine and amplitude are off by a few 2^-24 each
    and the fp32 products and sum by 2^-24 each: 2^-21 of (|a| + |b|) * amplitude covers them."""
    want = rope_ref(x, pos, freqs, rot, **kw)
    amp = abs(kw.get("amplitude", 1.0))
    size = rope_ref(x.abs(), torch.zeros_like(pos), freqs, rot, interleaved=kw.get("interleaved", False),
                    sections=kw.get("sections"))
    if kw.get("interleaved"):
        other = size[..., :rot].reshape(*size.shape[:-1], rot // 2, 2).flip(-1).reshape(*size.shape[:-1], rot)
    else:
        other = size[..., :rot].roll(rot // 2, -1)
    tol = HALF_STEP[x.dtype] * want.abs() + 1e-30
    if x.dtype == torch.float16:
        tol += 2.0 ** -25                                   # half a step of its subnormals
    tol[..., :rot] += 2.0 ** -21 * amp * (size[..., :rot] + other) * (1 + HALF_STEP[x.dtype])
    assert ((y.double() - want).abs() - tol).max() <= 0
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (64, 64), (16, 16), (80, 48), (144, 144), (256, 256), (256, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_packed_tokens(libsa, cuda_ok, dtype, d, rot, interleaved):
    gen = torch.Generator("cuda").manual_seed(d + rot)
    for T, Hq, Hk in ((1, 1, 1), (37, 5, 2), (130, 40, 8)):
        q, k = (torch.randn(T, h, d, device="cuda", generator=gen).to(dtype) for h in (Hq, Hk))
        pos = torch.randint(-5, 1 << 20, (T,), device="cuda", generator=gen).to(torch.int32)
        freqs, amp = libsa.sa_rope_frequencies(rot, scaling="ramp", factor=4.0, original_len=8192)
        yq, yk = libsa.sa_rope(q, k, pos, freqs, rot=rot, interleaved=interleaved, amplitude=amp)
        _check(yq, q, pos, freqs, rot, interleaved=interleaved, amplitude=amp)
        _check(yk, k, pos, freqs, rot, interleaved=interleaved, amplitude=amp)
        only = libsa.sa_rope(q, None, pos, freqs, rot=rot, interleaved=interleaved, amplitude=amp)
        assert torch.equal(only, yq)


@pytest.mark.parametrize("interleaved", [False, True])
def test_video_grid_axes_and_batches(libsa, cuda_ok, interleaved):
    """[B, H, N, d] with frame, row and column positions, a section of zero pairs among four."""
    gen = torch.Generator("cuda").manual_seed(3)
    B, H, N, d = 2, 3, 2 * 5 * 7, 128
    q, k = (torch.randn(B, H, N, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
    freqs, _ = libsa.sa_rope_frequencies(d)
    for sections in ([22, 21, 21], [0, 32, 30, 2], [64]):
        pos = torch.randint(0, 900, (len(sections), B, N), device="cuda", generator=gen).to(torch.int32)
        yq, yk = libsa.sa_rope(q, k, pos, freqs, interleaved=interleaved, sections=sections)
        _check(yq, q, pos, freqs, d, interleaved=interleaved, sections=sections)
        _check(yk, k, pos, freqs, d, interleaved=interleaved, sections=sections)
        shared = libsa.sa_rope(q, None, pos[:, 0].contiguous(), freqs, interleaved=interleaved, sections=sections)
        _check(shared, q, pos[:, :1].expand(-1, B, -1), freqs, d, interleaved=interleaved, sections=sections)


def test_strides_in_place_and_the_rest_untouched(libsa, cuda_ok):
    """q and k as slices of a fused projection, rotated where they are: v stays as it was."""
    gen = torch.Generator("cuda").manual_seed(4)
    T, Hq, Hk, d, rot = 77, 6, 2, 64, 32
    qkv = torch.randn(T, Hq + 2 * Hk, d, device="cuda", generator=gen).half()
    was = qkv.clone()
    q, k, v = qkv.split([Hq, Hk, Hk], 1)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    freqs, _ = libsa.sa_rope_frequencies(rot)
    libsa.sa_rope(q, k, pos, freqs, rot=rot, out=(q, k))
    _check(q, was[:, :Hq], pos, freqs, rot)
    _check(k, was[:, Hq:Hq + Hk], pos, freqs, rot)
    assert torch.equal(v, was[:, Hq + Hk:])
    # transposed memory: [B, H, N, d] seen through [B, N, H, d]
    x = torch.randn(2, 9, 4, d, device="cuda", generator=gen).bfloat16().transpose(1, 2)
    y = libsa.sa_rope(x, None, pos[:9].contiguous(), freqs, rot=rot)
    _check(y, x, pos[:9].expand(2, 9), freqs, rot)


def test_inverse_is_the_transposed_map(libsa, cuda_ok):
    """<R x, g> = <x, R' g> and, with amplitude 1, R' R x = x; R' is also what differences of
    <R x, g> give."""
    gen = torch.Generator("cuda").manual_seed(5)
    T, H, d = 19, 3, 64
    x, g = (torch.randn(T, H, d, device="cuda", generator=gen) for _ in range(2))
    pos = torch.randint(0, 5000, (T,), device="cuda", generator=gen).to(torch.int32)
    freqs, _ = libsa.sa_rope_frequencies(48)
    back = libsa.sa_rope(g, None, pos, freqs, rot=48, amplitude=1.25, inverse=True)
    _check(back, g, pos, freqs, 48, amplitude=1.25, inverse=True)
    f = lambda z: (libsa.sa_rope(z, None, pos, freqs, rot=48, amplitude=1.25).double() * g.double()).sum().item()  # noqa: E731
    e = torch.randn_like(x)
    # the map is linear: a difference of any step is exact but for fp32 rounding of T * H * d terms
    assert abs((f(x + e) - f(x - e)) / 2 - (e.double() * back.double()).sum().item()) < 1e-3
    once = libsa.sa_rope(x, None, pos, freqs, rot=48)
    assert (libsa.sa_rope(once, None, pos, freqs, rot=48, inverse=True) - x).abs().max() < 2e-6 * x.abs().max() * 2


def test_empty_and_feeding_attention(libsa, cuda_ok):
    freqs, _ = libsa.sa_rope_frequencies(128)
    x = torch.zeros(0, 4, 128, device="cuda", dtype=torch.bfloat16)
    assert libsa.sa_rope(x, None, torch.zeros(0, device="cuda", dtype=torch.int32), freqs).shape == x.shape
    # scores of rotated q and k depend on distances alone: shifting all positions changes sa_attn_fwd little
    gen = torch.Generator("cuda").manual_seed(6)
    q, k, v = (torch.randn(1, 2, 200, 128, device="cuda", generator=gen).bfloat16() for _ in range(3))
    pos = torch.arange(200, device="cuda", dtype=torch.int32)
    near, far = (libsa.sa_attn_fwd(*libsa.sa_rope(q, k, pos + off, freqs), v).float() for off in (0, 1 << 19))
    assert torch.nn.functional.cosine_similarity(near.flatten(), far.flatten(), 0) > 0.999
    assert libsa.sa_get_device_status() == 0
