"""A stricter 64-bit check of attention over the cache (not collected): NaN has to agree in both
outputs, and the bound of o is relative to what the row sees, with no absolute part."""
import math

import torch

from _cache_ref import HALF_STEP, PAGE


def attn_ref(cache, q, starts, lens, table, causal=True, window=0, sm_scale=None):
    """(o, lse, spread, most, reach, span, keys) in 64 bits.  For each row and head: spread is
    sum p |v| / l; most the largest weight times value scale, max p scale_v / l; reach the largest
    sum |q| |k| sm_scale; span the largest exponent that the weights are taken through; keys their number."""
    kc, ks, vc, vs = (t.double() for t in cache)
    T, Hq, d = q.shape
    H = kc.shape[1]
    G = Hq // H
    scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(o)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    most, reach, span, keys = (torch.zeros(T, Hq, dtype=torch.float64, device=q.device) for _ in range(4))
    starts, lens = starts.tolist(), lens.tolist()
    for b, length in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if n == 0 or length == 0:
            continue
        t = torch.arange(length, device=q.device)
        page, slot = table[b].long()[t // PAGE], t % PAGE
        p = torch.arange(length - n, length, device=q.device)[:, None]
        sees = (p >= 0) & (t >= 0)
        if causal:
            sees = sees & (t <= p)
        if window > 0:
            sees = sees & (t > p - window)
        rows = slice(starts[b], starts[b + 1])
        for h in range(H):
            cols = slice(h * G, (h + 1) * G)
            k, v = kc[page, h, slot] * ks[page, h][:, None], vc[page, h, slot] * vs[page, h][:, None]
            qq = q[rows, cols].double()
            x = (torch.einsum("ngd,td->ngt", qq, k) * scale).masked_fill(~sees[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            w = torch.where(sees[:, None], torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
            l = w.sum(-1)
            ok = ~(l == 0)
            den = torch.where(ok, l, 1.0)
            bad = torch.isnan(v).any(1)                                   # reaches the rows that see it
            vz = torch.where((sees.any(0) & ~bad)[:, None], v, 0.0)
            o[rows, cols] = torch.einsum("ngt,td->ngd", w, vz) / den[..., None]
            o[rows, cols] = torch.where((sees & bad).any(1)[:, None, None], math.nan, o[rows, cols])
            spread[rows, cols] = torch.einsum("ngt,td->ngd", w, vz.abs()) / den[..., None]
            lse[rows, cols] = torch.where(ok, torch.log(den) + m[..., 0], -math.inf)
            svz = torch.where(sees.any(0) & ~bad, vs[page, h], 0.0)
            most[rows, cols] = (w * svz).amax(-1) / den
            reach[rows, cols] = torch.where(sees[:, None], torch.einsum("ngd,td->ngt", qq.abs(), k.abs()), 0.0).amax(-1) * scale
            log = torch.where(svz > 0, torch.log2(svz.clamp(min=1e-300)), 0.0).abs()
            span[rows, cols] = (torch.where(sees, log, 0.0).amax(-1))[:, None] * 2 + 24.0
            keys[rows, cols] = sees.sum(-1)[:, None].double()
    return o, lse, spread, most, reach, span, keys


def check(got, want, dtype):
    """|o - o_ref| within
      half a step of the output;
      2^-11 of each weight: its rounding to fp16;
      half a step of fp16's subnormals, 2^-25, for each key's weight, which is kept at least 2^6
        times its share of the row's largest weight times value scale, and codes up to 127;
      the scores' own error, a factor of the weights: fp32 sums of d products, off by at most 2^-19
        of the sum of magnitudes, and the roundings of exponents up to span (in powers of two), three
        of 2^-24 each in o and in l; 2^-20 for exp2 and the sums."""
    (o, lse), (ro, rlse, spread, most, reach, span, keys) = got, want
    assert torch.equal(torch.isnan(o), torch.isnan(ro)), "o: NaN elsewhere"
    size = rlse.abs()
    size = torch.where(torch.isfinite(size), size, 0.0)
    dx = 2.0 ** -19 * (reach + size) + 2.0 ** -20 + 2.0 ** -22 * span
    tol = HALF_STEP[dtype] * ro.abs() + (2.0 ** -11 + 2 * dx[..., None]) * spread + (2.0 ** -31 * 127 * keys * most)[..., None]
    tol = tol * (1 + 2.0 ** -10) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # second order; the type's own subnormals
    there = ~torch.isnan(ro)
    off = ((o.double() - ro).abs() - tol)[there]
    assert off.numel() == 0 or bool((off <= 0).all()), \
        f"o off by {((o.double() - ro).abs() / tol)[there].max().item():.3g} times its bound"
    if lse is not None:
        assert torch.equal(torch.isnan(lse), torch.isnan(rlse)), "lse: NaN elsewhere"
        empty = rlse == -math.inf
        assert torch.equal(lse == -math.inf, empty), "lse: -inf elsewhere"
        there = ~empty & ~torch.isnan(rlse)
        off = ((lse.double() - rlse).abs() - dx - 2.0 ** -24 * size)[there]
        assert off.numel() == 0 or bool((off <= 0).all()), f"lse off by {off.max().item():.3g} more than its bound"
