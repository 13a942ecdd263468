"""Writing and reading the cache for more sequences than a block of threads looks up at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _i32(t):
    return t.to(torch.int32).cuda()


@pytest.mark.parametrize("B", [255, 256, 257, 511, 513, 5000, 70000])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_each_token_finds_its_sequence(libsa, cuda_ok, B, most):
    """Sequences of 0 to `most` new tokens in empty caches, a few of them 64, one page each, in any
    order; rows before the first sequence and behind the last stay out of it."""
    gen = torch.Generator().manual_seed(B + most)
    H, d = 2, 64
    new = torch.randint(0, most + 1, (B,), generator=gen)
    new[::97] = 64
    starts = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]) + 5
    T = int(starts[-1]) + 70
    table = torch.randperm(B, generator=gen)[:, None]
    cache = libsa.sa_cache_alloc(B, H, d)
    k, v = (torch.randn(T, H, d, device="cuda").bfloat16() for _ in range(2))
    args = _i32(starts), _i32(new), _i32(table)
    libsa.sa_cache_append(cache, k, v, *args)
    got = libsa.sa_cache_read(cache, T, *args, dtype=torch.float32)
    assert libsa.sa_get_device_status() == 0
    seq = torch.repeat_interleave(torch.arange(B), new).cuda()
    slot = (torch.arange(5, T - 70) - torch.repeat_interleave(starts[:-1], new)).cuda()
    page = args[2][:, 0].long()[seq]
    for x, codes, scale, out in ((k, *cache[:2], got[0]), (v, *cache[2:], got[1])):
        x = x[5:T - 70].float()
        s = torch.zeros(B, H, device="cuda").index_reduce_(0, seq, x.abs().amax(2), "amax") / torch.tensor(127.0, device="cuda")
        assert torch.equal(scale[args[2][:, 0].long()], s)
        want = (x / s[seq][:, :, None]).round()
        assert torch.equal(codes[page, :, slot].float(), want)
        assert torch.equal(out[5:T - 70], want * s[seq][:, :, None])


def test_a_million_sequences(libsa, cuda_ok):
    """Most of them idle: the look-up of each is a few steps (seconds for each call if every token
    looked through all of them)."""
    B, H, d = 1 << 20, 4, 64
    busy = torch.tensor([0, 1, 77777, 524288, B - 1])
    new = torch.zeros(B, dtype=torch.long)
    new[busy] = torch.tensor([3, 1, 64, 10, 2])
    starts = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
    table = torch.full((B, 1), -1)
    table[busy, 0] = torch.tensor([4, 2, 0, 1, 3])
    args = _i32(starts), _i32(new), _i32(table)
    cache = libsa.sa_cache_alloc(5, H, d)
    k, v = (torch.randn(80, H, d, device="cuda").half() for _ in range(2))
    libsa.sa_cache_append(cache, k, v, *args)                           # to warm up
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    libsa.sa_cache_append(cache, k, v, *args)
    got = libsa.sa_cache_read(cache, 80, *args, dtype=torch.float32)
    end.record()
    assert libsa.sa_get_device_status() == 0
    for x, y, scale in ((k, got[0], cache[1]), (v, got[1], cache[3])):
        page = _i32(torch.repeat_interleave(table[busy, 0], new[busy])).long()
        assert bool(((x.float() - y).abs() <= 0.5001 * scale[page][:, :, None]).all())
    assert begin.elapsed_time(end) < 1000


@pytest.mark.parametrize("B", [300, 2000])
@pytest.mark.parametrize("how", ["falling", "some", "random"])
def test_offsets_out_of_order(libsa, cuda_ok, B, how):
    """Whatever the offsets are, each page holds its own sequence's tokens or is as it was, and sequences
    whose offsets fall are reported."""
    gen = torch.Generator().manual_seed(B)
    H, d, T = 1, 64, 2 * B
    starts = torch.arange(B + 1) * 2
    if how == "falling":
        starts = starts.flip(0)
    elif how == "some":
        at = torch.randperm(B, generator=gen)[:20]
        starts[at] = torch.randint(0, T, (20,), generator=gen)
    else:
        starts = torch.randint(-5, T + 5, (B + 1,), generator=gen)
    new = starts[1:] - starts[:-1]
    valid = (starts[:-1] >= 0) & (new >= 0) & (starts[1:] <= T) & (new <= 64)
    lens = torch.where(valid, new, 1)                                   # a longer one would not fit its page
    args = _i32(starts), _i32(lens), _i32(torch.arange(B)[:, None])
    cache = libsa.sa_cache_alloc(B, H, d)
    cache[1].fill_(-1.0)
    k = torch.randn(T, H, d, device="cuda").half()
    libsa.sa_cache_append(cache, k, k, *args)
    assert libsa.sa_get_device_status() == 8
    written = 0
    for b in (cache[1][:, 0] != -1).nonzero()[:, 0].tolist():
        if not valid[b]:
            # only the last of its tokens is in the cache, as its length says, or none of another's
            assert lens[b] == 1 and new[b] > 64 and starts[b] >= 0 and starts[b + 1] <= T
            x = k[starts[b + 1] - 1:starts[b + 1], 0].float()
        else:
            x = k[starts[b]:starts[b + 1], 0].float()
        s = x.abs().max() / torch.tensor(127.0, device="cuda")
        assert cache[1][b, 0] == s and torch.equal(cache[0][b, 0, :x.shape[0]].float(), (x / s).round())
        written += 1
    assert written == 0 if how == "falling" else written > B // 2 if how == "some" else True
