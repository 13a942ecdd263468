"""Calls over the cache whose work is past what the kernels count."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_no_workspace_for_refused_sizes(libsa, cuda_ok):
    """Sizes that the attention call refuses need 0 bytes, also where products of them overflow."""
    f = libsa.raw_library().sa_cache_attn_workspace_bytes
    assert f(1 << 20, 16, 8, 4, 128) > 0 and f(0, 1, 1, 1, 64) > 0
    for sizes in [((1 << 30) + 1, 1, 1, 1, 128), (1 << 62, 1, 8, 1 << 20, 128), (1 << 62, 1, 1, 4, 64),
                  (64, (1 << 20) + 1, 1, 1, 128), (64, 1 << 20, 8192, 1, 128), (64, 1, 65536, 1, 64), (64, 1, 256, 256, 64),
                  (1 << 20, 1, 1, 2048, 64), (1 << 29, 1, 33, 1, 64), (64, 1, 8, 0, 64), (64, 1, 8, 1, 96), (64, 0, 8, 1, 64)]:
        assert f(*sizes) == 0, sizes


def test_more_blocks_than_a_worker_counts(libsa, cuda_ok):
    """Two sequences of 2^30 tokens on one shared page, 60000 heads: 2^41 blocks of keys, hours of
    work, are left out and reported; a shorter call over the same cache is answered."""
    H, d, pages = 60000, 64, 1 << 24
    cache = tuple(torch.ones(s, device="cuda", dtype=t) for s, t in
                  [((1, H, 64, d), torch.int8), ((1, H), torch.float32)] * 2)
    table = torch.zeros(2, pages, device="cuda", dtype=torch.int32)
    q = torch.ones(2, H, d, device="cuda", dtype=torch.bfloat16)
    starts = torch.tensor([0, 1, 2], device="cuda", dtype=torch.int32)
    out = torch.full_like(q, 5.0)
    for length, status, value in ((64 * pages, 8, 5.0), (100, 0, 1.0)):
        lens = torch.full((2,), length, device="cuda", dtype=torch.int32)
        libsa.sa_cache_attn(cache, q, starts, lens, table, out=out)
        assert libsa.sa_get_device_status() == status
        assert (out == value).all()
