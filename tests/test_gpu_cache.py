"""Writing and reading the paged INT8 cache, bit for bit against the definition: blocks that
grow, ragged batches, padding, strides, non-finite values, bad pages, large caches."""
import numpy as np
import pytest
import torch

from _cache_ref import append_ref, random_cache, random_table, starts_of

pytestmark = pytest.mark.gpu


def _host(cache):
    return [t.cpu().numpy() for t in cache]


def _same(got, want):
    for g, w in zip(got, want):
        assert g.dtype == w.dtype and np.array_equal(g, w, equal_nan=g.dtype.kind == "f"), np.argwhere(g != w)[:4]


def _append_and_check(libsa, cache, k, v, new, lens, table):
    starts, tab = np.concatenate([[0], np.cumsum(new)]), table.cpu().numpy()
    kc, ks, vc, vs = _host(cache)
    libsa.sa_cache_append(cache, k, v, starts_of(new), torch.tensor(lens, dtype=torch.int32, device="cuda"), table)
    assert libsa.sa_get_device_status() == 0
    want = [*append_ref(kc, ks, k.cpu().double().numpy(), starts, lens, tab),
            *append_ref(vc, vs, v.cpu().double().numpy(), starts, lens, tab)]
    _same(_host(cache), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", [1, 5])
def test_ragged_batches(libsa, cuda_ok, d, dtype, H):
    """New pieces that begin and end anywhere in a block; every other page keeps its bytes."""
    gen = torch.Generator().manual_seed(d + H)
    new, lens = [1, 64, 63, 0, 200, 1, 130, 65, 1], [1, 64, 127, 77, 201, 64, 700, 65, 129]
    cache = random_cache(gen, 60, H, d)
    table = random_table(gen, lens, 60, extra=2)
    k, v = (torch.randn(sum(new), H, d, generator=gen).cuda().to(dtype) for _ in range(2))
    _append_and_check(libsa, cache, 8 * k, v, new, lens, table)


def test_rounding_of_quotients(libsa, cuda_ok):
    """Many values, maxima of every kind: each code is the rounded fp32 quotient's (ties at
    x = max / 2 among them), from the smallest subnormals to the largest numbers."""
    gen = torch.Generator().manual_seed(8)
    H, d, T = 16, 128, 64 * 40
    x = torch.randn(T, H, d, generator=gen)
    x[:, :, ::9] = (x.reshape(40, 64, H, d).abs().amax((1, 3))[:, None, :, None] / 2).expand(40, 64, H, d).reshape(T, H, d)[:, :, ::9]
    power = torch.linspace(-133, 126, 40).round().repeat_interleave(64)[:, None, None]
    big = torch.ldexp(x.double(), power.double()).float().clamp(-3.3e38, 3.3e38)
    cache = random_cache(gen, 40, H, d)
    _append_and_check(libsa, cache, big.cuda().bfloat16(), x.cuda().bfloat16(), [T], [T], random_table(gen, [T], 40))
    half = torch.ldexp(x.double(), power.double().clamp(-24, 12)).float().clamp(-6e4, 6e4)
    _append_and_check(libsa, cache, half.cuda().half(), x.cuda().half(), [T], [T], random_table(gen, [T], 40))


def test_token_by_token_growth_and_zeros(libsa, cuda_ok):
    """130 tokens one at a time with growing size: old codes are re-rounded as defined each
    time; a sequence of zeros keeps scale 0 until its first value."""
    gen = torch.Generator().manual_seed(9)
    H, d, B = 2, 64, 3
    lens = [130, 130, 130]
    cache, table = random_cache(gen, 12, H, d), random_table(gen, lens, 12)
    for t in range(130):
        k = torch.randn(B, H, d, generator=gen) * (1.0 + 0.3 * t)
        k[1] = 0.0 if t < 70 else k[1]
        k[2] *= 0.0 if t % 3 else -1.0
        v = torch.randn(B, H, d, generator=gen) * (5.0 / (1 + t))
        _append_and_check(libsa, cache, k.cuda().bfloat16(), v.cuda().bfloat16(), [1] * B, [t + 1] * B, table)


def test_padding_tokens_and_gaps(libsa, cuda_ok):
    """Idle rows (length 0), pieces that begin before the sequence, and tokens before the first
    or behind the last sequence: nothing is stored for them; they read as zero, or not at all."""
    gen = torch.Generator().manual_seed(10)
    H, d = 3, 128
    new, lens = [1, 5, 100, 1], [0, 3, 70, 9]
    cache, table = random_cache(gen, 12, H, d), random_table(gen, [1, 3, 70, 9], 12)
    k, v = (torch.randn(4 + 107 + 30, H, d, generator=gen).cuda().bfloat16() for _ in range(2))
    starts = 4 + starts_of(new)
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = _host(cache)
    libsa.sa_cache_append(cache, k, v, starts, dlens, table)
    st = np.concatenate([[0], np.cumsum(new)])
    tab = table.cpu().numpy()
    kk, vv = (t[4:].cpu().double().numpy() for t in (k, v))
    want = [*append_ref(*before[:2], kk, st, lens, tab), *append_ref(*before[2:], vv, st, lens, tab)]
    _same(_host(cache), want)
    outs = [torch.full((141, H, d), 7.0, device="cuda") for _ in range(2)]
    lib = libsa.raw_library()
    assert lib.sa_cache_read(outs[0].data_ptr(), outs[1].data_ptr(), 2, 141, starts.data_ptr(), dlens.data_ptr(),
                             table.data_ptr(), 4, table.shape[1], *[t.data_ptr() for t in cache], 12, H, d,
                             torch.cuda.current_stream().cuda_stream) == 0
    assert libsa.sa_get_device_status() == 0
    for side, out in enumerate(outs):
        out = out.cpu().numpy()
        assert (out[:4] == 7).all() and (out[111:] == 7).all()
        row = 4
        for b, n in enumerate(new):
            for i in range(n):
                p = lens[b] - n + i
                if p < 0:
                    assert (out[row] == 0).all()
                else:
                    page = tab[b][p // 64]
                    assert np.array_equal(out[row], want[2 * side][page, :, p % 64].astype(np.float32) *
                                          want[2 * side + 1][page][:, None])
                row += 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_read_rounds_once(libsa, cuda_ok, dtype, d):
    gen = torch.Generator().manual_seed(11)
    H, lens, new = 4, [300, 64, 1], [130, 64, 1]
    cache, table = random_cache(gen, 16, H, d), random_table(gen, lens, 16)
    k, v = libsa.sa_cache_read(cache, sum(new), starts_of(new), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               table, dtype=dtype)
    for out, codes, scale in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        row = 0
        for b, (n, length) in enumerate(zip(new, lens)):
            t = torch.arange(length - n, length, device="cuda")
            page = table[b].long()[t // 64]
            want = (codes[page, :, t % 64].float() * scale[page][:, :, None]).to(dtype)
            assert torch.equal(out[row:row + n], want)
            row += n


def test_strided_tokens_of_a_fused_projection(libsa, cuda_ok):
    gen = torch.Generator().manual_seed(12)
    H, d = 2, 128
    qkv = torch.randn(150, 4 * H, d, generator=gen).cuda().bfloat16()
    _, k, v = qkv.split([2 * H, H, H], 1)
    cache, lens = random_cache(gen, 8, H, d), [150]
    _append_and_check(libsa, cache, k, v, [150], lens, random_table(gen, lens, 8))
    with pytest.raises(ValueError):
        libsa.sa_cache_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), v, starts_of([150]),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), random_table(gen, lens, 8))


def test_non_finite_values_show(libsa, cuda_ok):
    """NaN or infinity in a block makes that block and head read as NaN, and nothing else; a
    new use of the page starts afresh."""
    gen = torch.Generator().manual_seed(13)
    H, d, lens = 2, 64, [256]
    cache, table = random_cache(gen, 4, H, d), random_table(gen, lens, 4)
    x = torch.randn(256, H, d, generator=gen).cuda().bfloat16()
    bad = x.clone()
    bad[70, 0, 3], bad[200, 1, 5] = float("nan"), float("-inf")
    st, dl = starts_of([256]), torch.tensor(lens, dtype=torch.int32, device="cuda")
    libsa.sa_cache_append(cache, bad, x, st, dl, table)
    k, v = libsa.sa_cache_read(cache, 256, st, dl, table, dtype=torch.float32)
    nan = torch.isnan(k).all(2)
    assert nan[64:128, 0].all() and nan[192:256, 1].all() and int(torch.isnan(k).any(2).sum()) == 128
    assert not torch.isnan(v).any()
    libsa.sa_cache_append(cache, x, x, st, dl, table)
    k2, _ = libsa.sa_cache_read(cache, 256, st, dl, table, dtype=torch.float32)
    assert not torch.isnan(k2).any() and torch.equal(k2, v)


def test_bad_pages_lengths_and_offsets_are_reported(libsa, cuda_ok):
    """Out-of-range indexes touch nothing, set the status, and leave the others' work intact."""
    gen = torch.Generator().manual_seed(14)
    H, d, pages = 2, 64, 6
    x = torch.randn(100, H, d, generator=gen).cuda().bfloat16()
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for starts, lens, tab, skipped in (
            (i32(0, 50, 100), i32(50, 50), i32(pages, 1, 2, 3).reshape(2, 2), {0}),
            (i32(0, 50, 100), i32(50, 50), i32(0, 1, -1, 3).reshape(2, 2), {1}),
            (i32(0, 50, 100), i32(129, 50), table, {0}),
            (i32(0, 50, 100), i32(-1, 50), table, {0}),
            (i32(0, 50, 101), i32(50, 50), table, {1})):
        cache = random_cache(gen, pages, H, d)
        was = _host(cache)
        libsa.sa_cache_append(cache, x, x, starts, lens, tab)
        assert libsa.sa_get_device_status() == 8 and libsa.sa_status_string(8) == "SA_ERR_BAD_INDEX"
        assert libsa.sa_get_device_status() == 0
        now = _host(cache)
        kept = [b for b in (0, 1) if b not in skipped]
        st = np.array([0, 50, 100])
        want = was[:2]
        for b in kept:
            want = append_ref(*want, x[st[b]:st[b + 1]].cpu().double().numpy(), [0, 50], [50], tab.cpu().numpy()[b:b + 1])
        _same(now[:2], want)
    k, _ = libsa.sa_cache_read(random_cache(gen, pages, H, d), 100, i32(0, 50, 100), i32(50, 50),
                               i32(0, 1, 99, 3).reshape(2, 2), dtype=torch.float32)
    assert torch.isnan(k[50:]).all() and not torch.isnan(k[:50]).any()
    assert libsa.sa_get_device_status() == 8


@pytest.mark.parametrize("tokens,B", [(150, 3), (20, 20)])
def test_offsets_out_of_order_are_reported(libsa, cuda_ok, tokens, B):
    """Offsets that jump ahead and back: the sequence beside the jump is reported and not stored,
    pages of no sequence stay as they were."""
    gen = torch.Generator().manual_seed(17)
    H, d, pages = 2, 128, 2 * B + 4
    x = torch.randn(tokens, H, d, generator=gen).cuda().bfloat16()
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").reshape(B, 2)
    lens = torch.full((B,), 128, dtype=torch.int32, device="cuda")
    for ahead in (10 ** 9, -10 ** 9, 100000):
        starts = torch.linspace(0, tokens, B + 1).to(torch.int32)
        starts[B // 2] = ahead
        starts = starts.cuda()
        cache = random_cache(gen, pages, H, d)
        was = [t.clone() for t in cache]
        libsa.sa_cache_append(cache, x, x, starts, lens, table)
        assert libsa.sa_get_device_status() == 8
        for t, w in zip(cache, was):
            assert torch.equal(t[2 * (B // 2):2 * (B // 2) + 2], w[2 * (B // 2):2 * (B // 2) + 2])
            assert torch.equal(t[2 * B:], w[2 * B:])
        libsa.sa_cache_read(cache, tokens, starts, lens, table)
        assert libsa.sa_get_device_status() == 8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_one_sequence_brings_all_the_tokens(libsa, cuda_ok, dtype):
    """A batch of few tokens on average, of which one sequence has all: over many blocks."""
    gen = torch.Generator().manual_seed(18)
    H, d, B = 3, 128, 80
    new = [0] * B
    new[33] = 300
    lens = [n + (7 * i) % 70 for i, n in enumerate(new)]
    cache, table = random_cache(gen, 160, H, d), random_table(gen, lens, 160)
    k, v = (torch.randn(300, H, d, generator=gen).cuda().to(dtype) for _ in range(2))
    _append_and_check(libsa, cache, k, v, new, lens, table)


def test_nothing_to_do(libsa, cuda_ok):
    cache = libsa.sa_cache_alloc(2, 2, 64)
    x = torch.zeros(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    libsa.sa_cache_append(cache, x, x, z(2), z(1), z(1, 1))
    assert libsa.sa_cache_read(cache, 0, z(2), z(1), z(1, 1))[0].shape == (0, 2, 64)
    assert libsa.sa_cache_attn(cache, x, z(2), z(1), z(1, 1)).shape == (0, 2, 64)
    assert libsa.sa_get_device_status() == 0


def test_many_sequences(libsa, cuda_ok):
    """More sequences than a block has threads, lengths 0 and up."""
    gen = torch.Generator().manual_seed(15)
    H, d, B = 1, 64, 700
    lens = [int(n) for n in torch.randint(0, 140, (B,), generator=gen)]
    new = [min(n, int(m)) for n, m in zip(lens, torch.randint(0, 3, (B,), generator=gen))]
    cache, table = random_cache(gen, 2200, H, d), random_table(gen, lens, 2200)
    k, v = (torch.randn(sum(new), H, d, generator=gen).cuda().half() for _ in range(2))
    _append_and_check(libsa, cache, k, v, new, lens, table)


def test_cache_beyond_32_bits(libsa, cuda_ok):
    """Codes beyond 4 GiB: the last pages of a large cache are written and read back."""
    H, d, pages = 8, 128, 67000
    cache = libsa.sa_cache_alloc(pages, H, d)
    assert cache[0].numel() > 1 << 32
    gen = torch.Generator().manual_seed(16)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(150, H, d, generator=gen).cuda().bfloat16() for _ in range(2))
    st, dl = starts_of([150]), torch.tensor([150], dtype=torch.int32, device="cuda")
    libsa.sa_cache_append(cache, k, v, st, dl, table)
    got = libsa.sa_cache_read(cache, 150, st, dl, table, dtype=torch.float32)
    small = libsa.sa_cache_alloc(3, H, d)
    tab = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    libsa.sa_cache_append(small, k, v, st, dl, tab)
    for g, w in zip(got, libsa.sa_cache_read(small, 150, st, dl, tab, dtype=torch.float32)):
        assert torch.equal(g, w)
    q = torch.randn(150, H, d, generator=gen).cuda().bfloat16()
    assert torch.equal(libsa.sa_cache_attn(cache, q, st, dl, table), libsa.sa_cache_attn(small, q, st, dl, tab))
    assert libsa.sa_get_device_status() == 0
