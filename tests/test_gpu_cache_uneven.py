"""Attention over the cache in batches of uneven sequences, with a check of lse that NaN fails: most
sequences bring a token, some a piece of a prompt, so that the kernel of few rows has several tiles of
one sequence and head, whole and last ones; and calls of all kinds under that check."""
import math

import pytest
import torch

import _cache_strict as strict
from _cache_ref import random_cache, random_table, starts_of

pytestmark = pytest.mark.gpu


def _case(seed, new, lens, H, G, d, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    lens = [int(n) for n in lens]
    pages = sum(-(-n // 64) for n in lens) + 3
    cache, table = random_cache(gen, pages, H, d), random_table(gen, [max(n, 1) for n in lens], pages + len(lens))
    table.clamp_(max=pages - 1)
    q = torch.randn(sum(new), H * G, d, generator=gen).cuda().to(dtype)
    return cache, q, starts_of(new), torch.tensor(lens, dtype=torch.int32, device="cuda"), table


def _run(libsa, case, **kw):
    got = libsa.sa_cache_attn(*case, return_lse=True, **kw)
    assert libsa.sa_get_device_status() == 0
    strict.check(got, strict.attn_ref(*case, **kw), case[1].dtype)
    return got


def _few(new, G):
    """Whether the call goes to the kernel of few rows (16 of a sequence and head on average)."""
    return sum(new) * G <= 16 * len(new) or len(new) > 4096


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 64, 300])
def test_a_piece_among_single_tokens(libsa, cuda_ok, d, dtype, G, causal, window):
    new = [1] * 30 + [150] + [1] * 29 + [33, 0]
    lens = [1 + 37 * i % 700 for i in range(30)] + [333] + [1 + 91 * i % 900 for i in range(29)] + [1033, 70]
    assert _few(new, G)
    _run(libsa, _case(G, new, lens, 2, G, d, dtype), causal=causal, window=window)


@pytest.mark.parametrize("G", [1, 2, 5])
def test_a_prompt_among_many_single_tokens(libsa, cuda_ok, G):
    """Over a hundred tiles of one sequence and head, from its first token on or behind others, and
    tokens before their sequence."""
    new = [1] * 200 + [1500] if G == 1 else [1] * 300 + [1500 // G]
    for before in (0, 700, -40):
        case = _case(7 + G, new, [1 + 13 * i % 500 for i in range(len(new) - 1)] + [new[-1] + before], 2, G, 128)
        assert _few(new, G)
        _run(libsa, case)
        _run(libsa, case, causal=False, window=99)


def test_long_pieces_among_more_sequences_than_the_other_kernel_takes(libsa, cuda_ok):
    new = [1] * 4200
    new[17], new[4100], new[2000:2100] = 700, 333, [0] * 100
    lens = [1 + 7 * i % 130 for i in range(4200)]
    lens[17], lens[4100] = 900, 333
    _run(libsa, _case(9, new, lens, 1, 2, 64, torch.float16))


@pytest.mark.parametrize("G", [1, 7])
def test_pieces_of_several_workers(libsa, cuda_ok, G):
    """Tiles of one sequence over so long a cache that each is cut among several warps, and joined."""
    new = [1] * 12 + [29]
    case = _case(11, new, [100 * i + 1 for i in range(12)] + [30011], 2, G, 128)
    assert _few(new, G) == (G == 1)
    first = _run(libsa, case)
    for _ in range(5):
        again = libsa.sa_cache_attn(*case, return_lse=True)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("new,lens,G", [
    ([1] * 8, [1, 2, 63, 64, 65, 128, 700, 3333], 1), ([1, 1], [70001, 5], 4), ([1] * 4, [0, 64, 0, 1], 16),
    ([2, 1, 300, 65, 129, 17], [2, 64, 300, 200, 1000, 4099], 3), ([280], [16000], 1), ([700, 513], [2500, 513], 2),
    ([90, 90, 0, 90], [0, 130, 64, 87], 2),
])
@pytest.mark.parametrize("kw", [dict(), dict(causal=False), dict(window=100)])
def test_calls_of_all_kinds(libsa, cuda_ok, new, lens, G, kw):
    """Whole and joined segments of both kernels, idle sequences, tokens before theirs."""
    for d, dtype in ((64, torch.bfloat16), (128, torch.float16)):
        _run(libsa, _case(13, new, lens, 2, G, d, dtype), **kw)


@pytest.mark.parametrize("new,length", [(1, 400), (1, 60000), (16, 400), (150, 400), (150, 20000)])
def test_nan_in_both_outputs(libsa, cuda_ok, new, length):
    """NaN queries and key scales reach o and lse of the rows that see them, value scales o alone."""
    cache, q, starts, lens, table = _case(17, [new], [length], 2, 1, 128)
    blk = length // 64 - 2
    bad = q.clone()
    bad[0, 1, 5] = math.nan
    _run(libsa, (cache, bad, starts, lens, table), window=130)
    for which in (1, 3):
        spoilt = [t.clone() for t in cache]
        spoilt[which][table[0, blk].long(), 0] = math.nan
        o, lse = _run(libsa, (spoilt, q, starts, lens, table), window=130)
        assert torch.isnan(o[-1, 0]).all() and torch.isnan(lse[-1, 0]) == (which == 1)
        assert not torch.isnan(o[:, 1]).any() and not torch.isnan(lse[:, 1]).any()


def test_the_check_sees_nan(libsa, cuda_ok):
    """The check fails where an output is NaN and the reference is not, and the other way round."""
    case = _case(19, [3], [100], 1, 2, 64)
    want = strict.attn_ref(*case)
    for i in (0, 1):
        got = [t.clone() for t in libsa.sa_cache_attn(*case, return_lse=True)]
        strict.check(got, want, case[1].dtype)
        got[i].view(-1)[3] = math.nan
        with pytest.raises(AssertionError, match="NaN elsewhere"):
            strict.check(got, want, case[1].dtype)
