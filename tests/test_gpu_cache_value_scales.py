"""Attention over blocks whose value scales are far apart: what a row does not see changes nothing
in it, and what it sees counts by its weight, however small or large its scale."""
import math

import pytest
import torch

import _cache_strict as strict
from _cache_ref import random_table, starts_of

pytestmark = pytest.mark.gpu

# new tokens, cached ones, query heads on each of the key/value heads: segments of the tensor-core
# kernel, and tiles of one and two times eight rows of the other one
MANY = [(300, 1000, 1), (1000, 1000, 2), (150, 700, 5)]
FEW = [(8, 196, 1), (16, 330, 1), (5, 1026, 3), (4, 66, 2)]


def _case(seed, n, length, G, d, dtype=torch.bfloat16, q_scale=1.0):
    """One sequence of two heads; of few rows so many of sixteen that each warp of the GPU has several
    blocks of a sequence, one after another."""
    blocks = -(-length // 64)
    B, H = (8000 // (16 * blocks), 16) if (n, length, G) in FEW else (1, 2)
    gen = torch.Generator("cuda").manual_seed(seed)
    pages = B * blocks + 3
    codes = [torch.randint(-127, 128, (pages, H, 64, d), generator=gen, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.rand((pages, H), generator=gen, device="cuda") * 0.04 + 0.005 for _ in range(2)]
    table = random_table(torch.Generator().manual_seed(seed), [length] * B, pages)
    q = (q_scale * torch.randn(B * n, H * G, d, generator=gen, device="cuda")).to(dtype)
    return ([codes[0], scale[0], codes[1], scale[1]], q, starts_of([n] * B),
            torch.tensor([length] * B, dtype=torch.int32, device="cuda"), table)


def _check(got, cache, q, starts, lens, table, causal=True, window=0):
    """Against 64 bits, the first three sequences."""
    rows = starts[:4][-1].item()
    want = strict.attn_ref(cache, q[:rows], starts[:4], lens[:3], table[:3], causal, window)
    strict.check(tuple(t[:rows] for t in got), want, q.dtype)


def _sees_block(n, length, blk, causal, window):
    """Whether the query at each of the n positions sees any token of the block."""
    p = torch.arange(length - n, length, device="cuda")
    first = (p - window + 1).clamp(min=0) if window else torch.zeros_like(p)
    last = p if causal else torch.full_like(p, length - 1)
    return (first < 64 * blk + 64) & (last >= 64 * blk)


@pytest.mark.parametrize("n,length,G,causal,window", [
    (*shape, *mask) for shape in MANY for mask in [(True, 0), (True, 100), (False, 100), (True, 64)]] + [
    (*shape, True, 0) for shape in FEW] + [
    (*shape, causal, window) for causal in (True, False) for shape, window in zip(FEW, (64, 70, 192))])
@pytest.mark.parametrize("power", [20, 32, 60])
def test_blocks_that_a_row_does_not_see(libsa, cuda_ok, n, length, G, causal, window, power):
    """A block of 2^power times the others' value scale: rows that do not see it are the same, bit for
    bit, as without it; each block in turn of those that some new token sees and another does not."""
    cache, q, starts, lens, table = _case(n + G, n, length, G, 64 if G == 1 else 128)
    kw = dict(causal=causal, window=window, return_lse=True)
    clean = libsa.sa_cache_attn(cache, q, starts, lens, table, **kw)
    tried = 0
    for blk in range(-(-length // 64)):
        sees = _sees_block(n, length, blk, causal, window).repeat(lens.shape[0])
        if sees.all() or not sees.any():
            continue
        tried += 1
        vs = cache[3].clone()
        vs[table[:, blk].long()] *= 2.0 ** power
        got = libsa.sa_cache_attn((*cache[:3], vs), q, starts, lens, table, **kw)
        assert torch.equal(got[0][~sees], clean[0][~sees]), f"block {blk}"
        assert torch.equal(got[1][~sees], clean[1][~sees]), f"block {blk}"
        _check(got, (*cache[:3], vs), q, starts, lens, table, causal, window)
    assert tried > (n * G > 16) and libsa.sa_get_device_status() == 0


@pytest.mark.parametrize("n,length,G", MANY + FEW)
@pytest.mark.parametrize("weight", [-20, -32, -44, -100])
def test_a_large_block_of_little_weight(libsa, cuda_ok, n, length, G, weight):
    """A block of 2^32 times the value scale whose keys have about 2^weight of a row's weight: it
    decides the output, shares it, or disappears, as its product with the weight says."""
    d = 128
    cache, q, starts, lens, table = _case(7, n, length, G, d)
    q[:] = 1.0
    cache[1] *= 0.02  # the other scores are about 0
    page = table[:, length // 64 // 2].long()
    cache[0][page] = -127
    cache[1][page] = -weight * math.log(2.0) / (127 * math.sqrt(d))
    cache[3][page] *= 2.0 ** 32
    got = libsa.sa_cache_attn(cache, q, starts, lens, table, return_lse=True)
    _check(got, cache, q, starts, lens, table)


@pytest.mark.parametrize("n,length,G", MANY + FEW)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (False, 0), (False, 70)])
@pytest.mark.parametrize("spread", [8, 40, 90])
def test_scales_of_all_sizes(libsa, cuda_ok, n, length, G, causal, window, spread):
    """Each block and head its own value scale, up to 2^spread apart, zero ones among them, with
    sharp and with flat scores."""
    for q_scale in (0.3, 6.0):
        cache, q, starts, lens, table = _case(spread + n, n, length, G, 128, q_scale=q_scale)
        gen = torch.Generator("cuda").manual_seed(spread)
        cache[3] *= torch.pow(2.0, (torch.rand(cache[3].shape, generator=gen, device="cuda") - 0.5) * spread)
        cache[3][::7] = 0.0
        got = libsa.sa_cache_attn(cache, q, starts, lens, table, causal=causal, window=window, return_lse=True)
        _check(got, cache, q, starts, lens, table, causal, window)


@pytest.mark.parametrize("n,length,G", MANY + FEW)
@pytest.mark.parametrize("power", [-112, -60, 60, 112])
def test_scales_all_small_or_large(libsa, cuda_ok, n, length, G, power):
    cache, q, starts, lens, table = _case(11, n, length, G, 64)
    cache[3] *= 2.0 ** power
    got = libsa.sa_cache_attn(cache, q, starts, lens, table, return_lse=True)
    _check(got, cache, q, starts, lens, table)
