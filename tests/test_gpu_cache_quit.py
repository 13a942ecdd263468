"""A worker of the attention over the cache that gives up, as after an expired wait: the status says so,
what others join with its pieces is NaN, nothing else changes, and the next call is as before.  The
worker is told to stop by the host; no wait runs out and nothing faults."""
import pytest
import torch

from _cache_ref import random_cache, random_table, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture
def quits(libsa):
    yield libsa.raw_library().sa_debug_cache_attn_quit
    libsa.raw_library().sa_debug_cache_attn_quit(-1)


def _call(libsa, new, lens, H, d, dtype):
    gen = torch.Generator().manual_seed(5)
    pages = sum(-(-n // 64) for n in lens) + 3
    cache, table = random_cache(gen, pages, H, d), random_table(gen, lens, pages)
    q = torch.randn(sum(new), H, d, generator=gen).cuda().to(dtype)
    starts, dlens = starts_of(new), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call():
        out = torch.full_like(q, 5.0)
        return libsa.sa_cache_attn(cache, q, starts, dlens, table, causal=False, return_lse=True, out=out)
    return call


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("new", [1, 10, 100, 256])
def test_pieces_of_one_sequence(libsa, cuda_ok, quits, new, d, dtype):
    """One segment that all workers share: the first has nothing joined, another's piece spoils it."""
    call = _call(libsa, [new], [20001], 1, d, dtype)
    good = call()
    for _ in range(3):
        for worker, left in ((0, True), (7, False), (20, False)):
            quits(worker)
            o, lse = call()
            assert libsa.sa_get_device_status() == 6
            assert (o == 5).all() if left else torch.isnan(o).all() and torch.isnan(lse).all()
            quits(-1)
            again = call()
            assert libsa.sa_get_device_status() == 0
            assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("new,B,H", [(1, 3000, 2), (40, 300, 3)])
def test_others_are_untouched(libsa, cuda_ok, quits, new, B, H, d, dtype):
    """Many short sequences: only those of the worker are left out or NaN, a few of them."""
    call = _call(libsa, [new] * B, [40 + 64 * (i % 3) for i in range(B)], H, d, dtype)
    good = call()
    seen = set()
    for worker in (0, 1, 50, 130):
        quits(worker)
        o, lse = call()
        assert libsa.sa_get_device_status() == 6
        lost = torch.isnan(o).all(2) | (o == 5).all(2)                   # [tokens, heads]
        assert torch.equal(o[~lost], good[0][~lost]) and torch.equal(lse[~lost], good[1][~lost])
        assert torch.isnan(lse[torch.isnan(o).all(2)]).all()
        assert 0 < lost.sum() < lost.numel() // 20
        seen.add(tuple(lost.nonzero()[0].tolist()))
    assert len(seen) == 4
    quits(-1)
    assert torch.equal(call()[0], good[0]) and libsa.sa_get_device_status() == 0
