"""Plain 64-bit references of the rotary code, the paged INT8 cache and attention over it, and
builders of their inputs (not collected).  Written from the definitions in include/sa.h."""
import math

import numpy as np
import torch

PAGE = 64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # eps / 2


def fl(x):
    """One rounding to fp32."""
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def append_ref(codes, scale, x, starts, lens, table):
    """numpy codes int8 [pages, H, 64, d], scale fp32 [pages, H] after appending x fp64 [T, H, d]."""
    codes, scale = codes.copy(), scale.astype(np.float64)
    for b, length in enumerate(lens):
        n = starts[b + 1] - starts[b]
        start = length - n
        for j in range(max(start, 0) // PAGE, -(-length // PAGE)):
            lo, hi = max(start, 0, PAGE * j), min(length, PAGE * j + PAGE)
            if lo >= hi:
                continue
            page, old = table[b][j], lo - PAGE * j
            new = x[starts[b] + lo - start:starts[b] + hi - start]
            for h in range(x.shape[1]):
                s = fl(np.abs(new[:, h]).max() / 127.0)
                if old:
                    was = scale[page, h]
                    s = max(s, was)
                    r = fl(was / s) if s > 0 else 0.0
                    if s != was:
                        codes[page, h, :old] = np.rint(fl(codes[page, h, :old].astype(np.float64) * r))
                c = np.rint(fl(new[:, h] / s)) if s > 0 else np.zeros_like(new[:, h])
                codes[page, h, old:old + hi - lo] = np.clip(c, -127, 127)
                scale[page, h] = s
    return codes, scale.astype(np.float32)


def random_cache(gen, pages, H, d, device="cuda", shift=1.0):
    """A cache of random codes and scales (every page holds something)."""
    kc, vc = (torch.randint(-127, 128, (pages, H, PAGE, d), generator=gen, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand((pages, H), generator=gen) * 0.04 + 0.005 for _ in range(2))
    return tuple(t.to(device) for t in (kc, ks * shift, vc, vs))


def random_table(gen, lens, pages, extra=0, device="cuda"):
    """Distinct random pages for every block; unused entries are out of range on purpose."""
    need = [-(-n // PAGE) for n in lens]
    order = torch.randperm(pages, generator=gen)[:sum(need)].to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + extra), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(device)


def starts_of(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")


def attn_ref(cache, q, starts, lens, table, causal=True, window=0, sm_scale=None):
    """(o, lse, spread, reach): fp64 attention; spread is sum p |v| / l and reach the largest
    sum |q| |k| * sm_scale of a row's scores, for error bounds."""
    kc, ks, vc, vs = (t.double() for t in cache)
    T, Hq, d = q.shape
    H = kc.shape[1]
    G = Hq // H
    scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(o)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros(T, Hq, dtype=torch.float64, device=q.device)
    starts, lens = starts.tolist(), lens.tolist()
    for b, length in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if n == 0 or length == 0:
            continue
        t = torch.arange(length, device=q.device)
        page, slot = table[b].long()[t // PAGE], t % PAGE
        p = torch.arange(length - n, length, device=q.device)[:, None]
        sees = torch.ones(n, length, dtype=torch.bool, device=q.device) & (p >= 0)
        if causal:
            sees &= t <= p
        if window > 0:
            sees &= t > p - window
        rows = slice(starts[b], starts[b + 1])
        for h in range(H):
            k, v = kc[page, h, slot] * ks[page, h][:, None], vc[page, h, slot] * vs[page, h][:, None]
            qq = q[rows, h * G:(h + 1) * G].double()                       # [n, G, d]
            x = torch.einsum("ngd,td->ngt", qq, k) * scale
            x = x.masked_fill(~sees[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
            l = w.sum(-1)
            ok = l > 0
            den = torch.where(ok, l, 1.0)[..., None]
            vz = torch.where(sees.any(0)[:, None], v, 0.0)                 # unseen by every row: 0 * NaN
            o[rows, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w, vz) / den
            spread[rows, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w, vz.abs()) / den
            lse[rows, h * G:(h + 1) * G] = torch.where(ok, torch.log(den[..., 0]) + m[..., 0], -math.inf)
            reach[rows, h * G:(h + 1) * G] = torch.einsum("ngd,td->ngt", qq.abs(), k.abs()).amax(-1) * scale
    return o, lse, spread, reach


def check_attn(got, want, dtype):
    """|o - o_ref| within: half a step of the output; half a step of fp16 (2^-11) for each
    softmax weight; the scores' own error, whose fp32 sums of d products are off by at most
    2^-19 of the sum of magnitudes (d / 16 accumulations of 2^-23, products and scales a few
    2^-24) and enter the weights as a factor; 2^-20 for exp2 and the sums."""
    (o, lse), (ro, rlse, spread, reach) = got, want
    assert torch.equal(torch.isnan(o), torch.isnan(ro).to(o.device))
    dx = 2.0 ** -19 * (reach + rlse.abs().clamp(max=1e30).nan_to_num(0.0)) + 2.0 ** -20
    tol = HALF_STEP[dtype] * ro.abs() + (2.0 ** -11 + 2 * dx[..., None]) * spread + 2.0 ** -24
    off = ((o.double() - ro).abs() - tol).nan_to_num(-1.0)
    assert off.max() <= 0, f"o off by {off.max().item()} more than its bound"
    if lse is not None:
        empty = rlse == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        e = ((lse.double() - rlse).abs() - dx)[~empty].nan_to_num(-1.0)
        assert e.numel() == 0 or e.max() <= 0, f"lse off by {e.max().item()} more than its bound"


def rope_ref(x, pos, freqs, rot, interleaved=False, sections=None, amplitude=1.0, inverse=False):
    """fp64 rotation of x [B, H, N, d] or [T, H, d]; pos with the axes in front if sections."""
    y = x.double().clone()
    p = pos.double()
    axis = torch.zeros(rot // 2, dtype=torch.long) if sections is None else \
        torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    for i in range(rot // 2):
        f = (p if sections is None else p[axis[i]]) * freqs[i]
        c, s = amplitude * torch.cos(f), amplitude * torch.sin(f) * (-1 if inverse else 1)
        if x.dim() == 3:
            c, s = c[:, None], s[:, None]
        else:
            c, s = (t.reshape(-1, 1, x.shape[2]) for t in (c, s))
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., u].double(), x[..., w].double()
        y[..., u], y[..., w] = a * c - b * s, b * c + a * s
    return y
