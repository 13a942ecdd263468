"""The serving operators of the library, what they are measured on, and their plain forms.

Four operators make up a step of generation over a cache held in 8 bits:
  rope    rotary positions of queries and keys (sa_rope);
  append  new keys and values into a paged INT8 cache with one scale for each block of 64
          tokens and head (sa_cache_append), followed by reading the touched blocks back
          (sa_cache_read), which is how a program sees what the cache now stands for;
  decode  attention of single tokens over that cache (sa_cache_attn);
  chunk   attention of many tokens of each sequence over it (sa_cache_attn).

`listed()` has the measured cases and `draw(rng)` gives more of the same ranges.
`prepare(case, seed)` makes the inputs, `run(state)` is one pass: the library's entry points
where the module's `own` is true, elementary torch operations in 32 bits otherwise (64 for the
angles).  `exact(case, seed)` evaluates the definitions in 64 bits.

Definitions.  A block is 64 consecutive tokens of one sequence, token t lies in block t // 64.
  rope:   (a, b) -> amplitude * (a cos f - b sin f, b cos f + a sin f), f = pos * freqs[i], for
          pair i = channels (i, i + rot/2), or (2i, 2i + 1) interleaved; other channels unchanged.
  append: over the new tokens of a block and head, s_new = fl(max|x| / 127); with older tokens
          in the block s = max(s_old, s_new) and their codes become rint(fl(c * fl(s_old / s)));
          new codes are rint(fl(x / s)), within +-127 (fl: one rounding to 32 bits; s = 0: 0).
  read:   scale * code.
  attn:   query i of the n of a sequence with L cached tokens stands at p = L - n + i and sees
          the tokens t < L with t <= p (causal) and t > p - window (if window > 0):
          o = sum softmax(q.k * sm_scale) v, lse = log sum exp(q.k * sm_scale).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One decoding step of a batch: few rows, so the launch itself counts.
        {"name": "rope-step", "op": "rope", "dtype": "bf16", "batch": 0, "tokens": 64, "q_heads": 40, "k_heads": 8,
         "d": 128, "rot": 128, "interleaved": False, "axes": 1, "far": 1 << 20, "fused": False},
        # The whole latent grid of a 480p video (21 x 30 x 52), rotated by frame, row and column.
        {"name": "rope-video", "op": "rope", "dtype": "bf16", "batch": 1, "tokens": 32760, "q_heads": 12, "k_heads": 12,
         "d": 128, "rot": 128, "interleaved": True, "axes": 3, "far": 0, "fused": False},
        # A prompt taken out of a fused projection, half of each head rotated, long context.
        {"name": "rope-prompt-part", "op": "rope", "dtype": "fp16", "batch": 0, "tokens": 10007, "q_heads": 32,
         "k_heads": 4, "d": 64, "rot": 32, "interleaved": False, "axes": 1, "far": 1 << 17, "fused": True},
        # One token more for each of 64 sequences, most of them into a partly filled block.
        {"name": "append-step", "op": "append", "dtype": "bf16", "batch": 64, "new": 1, "lo": 65, "hi": 2500, "heads": 8,
         "d": 128, "fused": False},
        # The tokens of one latent frame (30 x 52) behind 20 cached ones.
        {"name": "append-frame", "op": "append", "dtype": "bf16", "batch": 1, "new": 1560, "lo": 32760, "hi": 32760,
         "heads": 40, "d": 128, "fused": False},
        # Whole prompts of odd lengths from a fused projection.
        {"name": "append-prompts", "op": "append", "dtype": "fp16", "batch": 5, "new": 0, "lo": 301, "hi": 20011,
         "heads": 16, "d": 64, "fused": True},
        # One sequence, a short cache: nothing but latency.
        {"name": "decode-short", "op": "decode", "dtype": "bf16", "batch": 1, "lo": 1000, "hi": 1000, "q_heads": 12,
         "k_heads": 12, "d": 128, "window": 0, "fused": False},
        # A serving batch of ragged lengths with shared heads.
        {"name": "decode-batch", "op": "decode", "dtype": "bf16", "batch": 64, "lo": 1, "hi": 8192, "q_heads": 40,
         "k_heads": 8, "d": 128, "window": 0, "fused": True},
        # A few very long sequences.
        {"name": "decode-long", "op": "decode", "dtype": "fp16", "batch": 4, "lo": 70001, "hi": 131072, "q_heads": 32,
         "k_heads": 8, "d": 128, "window": 0, "fused": False},
        # Short ragged chunks with a sliding window and small heads.
        {"name": "chunk-window", "op": "chunk", "dtype": "fp16", "batch": 6, "new_lo": 17, "new_hi": 400, "lo": 401,
         "hi": 3001, "q_heads": 8, "k_heads": 2, "d": 64, "causal": True, "window": 512, "fused": False},
        # Prompts in pieces over their earlier pieces, causal, shared heads.
        {"name": "chunk-prompts", "op": "chunk", "dtype": "bf16", "batch": 2, "new_lo": 1901, "new_hi": 2048, "lo": 6001,
         "hi": 8192, "q_heads": 32, "k_heads": 4, "d": 128, "causal": True, "window": 0, "fused": True},
        # One latent frame that sees every cached frame and itself (40 heads, 480p).
        {"name": "chunk-frame", "op": "chunk", "dtype": "bf16", "batch": 1, "new_lo": 1560, "new_hi": 1560, "lo": 32760,
         "hi": 32760, "q_heads": 40, "k_heads": 40, "d": 128, "causal": False, "window": 0, "fused": False},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope", "append", "decode", "chunk"])
    d = rng.choice([64, 128])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "d": d}
    kh = rng.choice([1, 2, 3, 4, 5, 8, 10, 12, 16])
    if op == "rope":
        grid = rng.random() < 0.4
        case.update(batch=rng.choice([1, 2]) if grid else 0, tokens=log(1, 16000), q_heads=kh * rng.choice([1, 2, 5]),
                    k_heads=rng.choice([0, kh]), rot=rng.choice([16, 32, 48, d]), interleaved=rng.random() < 0.5,
                    axes=3 if grid else 1, far=log(1, 1 << 20), fused=not grid and rng.random() < 0.5)
    elif op == "append":
        one = rng.random() < 0.5
        batch = log(1, 200) if one else rng.randint(1, 6)
        hi = log(1, 3000) if one else log(1, 60000 // batch)
        lo = rng.randint(1, hi)
        case.update(batch=batch, new=1 if one else rng.choice([0, rng.randint(1, lo)]), lo=lo, hi=hi, heads=kh,
                    fused=rng.random() < 0.5)
    elif op == "decode":
        batch = log(1, 128)
        hi = log(1, min(131072, 3000000 // (batch * kh)))
        case.update(batch=batch, lo=rng.randint(1, hi), hi=hi, q_heads=kh * rng.choice([1, 2, 3, 4, 5, 8, 16]),
                    k_heads=kh, window=rng.choice([0, 0, log(1, 4096)]), fused=rng.random() < 0.5)
    else:
        batch = rng.randint(1, 6)
        group = rng.choice([1, 1, 2, 3, 4, 8])
        new_hi = log(2, 1600)
        hi = new_hi + log(1, max(1, min(30000, 1500000000 // (batch * kh * group * new_hi))))
        new_lo = rng.randint(1, new_hi)
        case.update(batch=batch, new_lo=new_lo, new_hi=new_hi, lo=rng.randint(new_hi, hi), hi=hi, q_heads=kh * group,
                    k_heads=kh, causal=rng.random() < 0.6, window=rng.choice([0, 0, log(1, 4096)]),
                    fused=rng.random() < 0.5)
    return case


def _spread(lo, hi, n):
    """n whole numbers in [lo, hi], hi among them, spread without an order."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * (((i * 0.6180339887498949) + 0.3) % 1.0)) for i in range(n)]


def _kv_lens(case):
    """Cached tokens of each sequence, the new ones included."""
    return _spread(case["lo"], case["hi"], case["batch"])


def _new_lens(case):
    """New tokens (append, chunk) or query tokens (decode) of each sequence."""
    if case["op"] == "decode":
        return [1] * case["batch"]
    if case["op"] == "chunk":
        return _spread(case["new_lo"], case["new_hi"], case["batch"])
    return [n if case["new"] == 0 else case["new"] for n in _kv_lens(case)]


def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    return [half - 2 * (half // 3), half // 3, half // 3]


def _spans(case):
    """(query length, first and last seen token by query) of each sequence."""
    window, causal = case["window"], case.get("causal", True)
    for n, length in zip(_new_lens(case), _kv_lens(case)):
        p = np.arange(length - n, length)
        last = p if causal else np.full(n, length - 1)
        first = np.maximum(0, p - window + 1) if window > 0 else np.zeros(n, np.int64)
        yield n, first, last


def work(case):
    d, size = case["d"], 2
    if case["op"] == "rope":
        rows = max(1, case["batch"]) * case["tokens"]
        values = rows * (case["q_heads"] + case["k_heads"]) * d
        return {"bytes": 2 * size * values + 4 * case["axes"] * rows, "flops": 3 * values}
    if case["op"] == "append":
        new, lens = _new_lens(case), _kv_lens(case)
        kept = [(n - m) % PAGE for n, m in zip(lens, new)]
        values = sum(new) * case["heads"] * d
        seen = (sum(new) + sum(kept)) * case["heads"] * d
        # the new values in, their codes out; the touched blocks' codes in and their values out
        return {"bytes": 2 * (values * (size + 1) + seen * (1 + 4)), "flops": 2 * (4 * values + seen)}
    heads, kv = case["q_heads"], case["k_heads"]
    rows = sum(_new_lens(case))
    tokens = pairs = 0
    for _, first, last in _spans(case):
        tokens += int(last[-1] - first[0] + 1)
        pairs += int((last - first + 1).sum())
    return {"bytes": 2 * tokens * kv * d + 8 * kv * (tokens // PAGE) + 2 * size * rows * heads * d + 4 * rows * heads,
            "flops": 4 * pairs * heads * d}


# ------------------------------------------------------------------ inputs


def _packed(gen, rows, widths, d, dtype, fused, shifts):
    """Tensors [rows, widths[i], d], N(0, 1) plus a shift by head and channel; with `fused` they
    are slices of one projection's output."""
    parts = [torch.randn(rows, w, d, generator=gen, device="cuda") for w in widths]
    for part, s in zip(parts, shifts):
        if s:
            part += s * torch.randn(1, part.shape[1], d, generator=gen, device="cuda")
    if fused:
        return list(torch.cat(parts, 1).to(dtype).split(widths, 1))
    return [p.to(dtype) for p in parts]


def _cache(case, gen, heads):
    """A cache that holds every sequence's tokens, its pages in random order."""
    lens, d = _kv_lens(case), case["d"]
    pages = [-(-n // PAGE) for n in lens]
    total, widest = sum(pages), max(pages)
    order = torch.randperm(total + 3, generator=gen, device="cuda")[:total].to(torch.int32)
    table = torch.zeros(case["batch"], widest, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    cache = []
    for shift in (2.0, 0.0):  # keys have an offset by channel, values have none
        codes = torch.empty(total + 3, heads, PAGE, d, dtype=torch.int8, device="cuda")
        scale = torch.empty(total + 3, heads, device="cuda")
        off = shift * torch.randn(heads, 1, d, generator=gen, device="cuda")
        for i in range(0, total + 3, 512):
            x = torch.randn(min(512, total + 3 - i), heads, PAGE, d, generator=gen, device="cuda") + off
            s = x.abs().amax((2, 3)) / 127
            scale[i:i + 512] = s
            codes[i:i + 512] = (x / s[:, :, None, None]).round().clamp(-127, 127).to(torch.int8)
        cache += [codes, scale]
    return tuple(cache), table


def _starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dtype, d, op = _TYPES[case["dtype"]], case["d"], case["op"]
    state = {"case": dict(case)}
    if op == "rope":
        batch, n, rot = case["batch"], case["tokens"], case["rot"]
        widths = [case["q_heads"]] + ([case["k_heads"]] if case["k_heads"] else [])
        if batch:
            xs = [torch.randn(batch, w, n, d, generator=gen, device="cuda").to(dtype) for w in widths]
        else:
            xs = _packed(gen, n, widths, d, dtype, case["fused"], [0.0, 2.0])
        if case["axes"] == 3:
            # frame, row and column of a token of a latent grid, the frames from a random one on
            rows, cols = max(1, math.isqrt(n // 21)), max(1, n // 21 // max(1, math.isqrt(n // 21)))
            t = torch.arange(n, device="cuda")
            first = torch.randint(0, 4096, (1,), generator=gen, device="cuda")
            pos = torch.stack([t // (rows * cols) + first, t // cols % rows, t % cols]).to(torch.int32)
        else:
            rows = batch * n if batch else n
            pos = torch.randint(0, max(1, case["far"]), (rows,), generator=gen, device="cuda").to(torch.int32)
            pos = pos.reshape(batch, n) if batch else pos
        freqs = 1.0 / 10000.0 ** (torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        if case["far"] > 1 << 16:  # scaled for a long context
            freqs, state["amplitude"] = freqs / 8.0, 0.1 * math.log(8.0) + 1.0
        else:
            state["amplitude"] = 1.0
        state.update(q=xs[0], k=xs[1] if len(xs) > 1 else None, pos=pos, freqs=freqs, sections=_sections(case))
        return state
    new, lens = _new_lens(case), _kv_lens(case)
    heads = case["heads"] if op == "append" else case["k_heads"]
    state["cache"], state["table"] = _cache(case, gen, heads)
    state["starts"], state["lens"] = _starts(new), torch.tensor(lens, dtype=torch.int32, device="cuda")
    state["rows"], state["widest"] = sum(new), max(new)
    if op == "append":
        state["k"], state["v"] = _packed(gen, sum(new), [heads, heads], d, dtype, case["fused"], [2.0, 0.0])
        seen = [m + (n - m) % PAGE for n, m in zip(lens, new)]
        state["seen_starts"], state["seen"] = _starts(seen), sum(seen)
    else:
        widths = [case["q_heads"]] + ([heads, heads] if case["fused"] else [])
        state["q"] = _packed(gen, sum(new), widths, d, dtype, case["fused"], [0.0] * 3)[0]
        state["scale"] = 1.0 / math.sqrt(d)
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_rope(s):
    from bit_quantized_attention_sa_b200 import binding as sa
    c = s["case"]
    return sa.sa_rope(s["q"], s["k"], s["pos"], s["freqs"], rot=c["rot"], interleaved=c["interleaved"],
                      sections=s["sections"], amplitude=s["amplitude"])


def _own_append(s):
    from bit_quantized_attention_sa_b200 import binding as sa
    sa.sa_cache_append(s["cache"], s["k"], s["v"], s["starts"], s["lens"], s["table"])
    return sa.sa_cache_read(s["cache"], s["seen"], s["seen_starts"], s["lens"], s["table"], dtype=torch.float32)


def _own_attn(s):
    from bit_quantized_attention_sa_b200 import binding as sa
    c = s["case"]
    return sa.sa_cache_attn(s["cache"], s["q"], s["starts"], s["lens"], s["table"], causal=c.get("causal", True),
                            window=c["window"], sm_scale=s["scale"], return_lse=True)


_OWN = {"rope": _own_rope, "append": _own_append, "decode": _own_attn, "chunk": _own_attn}


def _turn(x, cos, sin, rot, interleaved):
    """x [..., d] in 32 bits, cos and sin broadcast over [..., rot / 2]."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    first, second = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = first, second
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = first, second
    return y


def _plain_rope(s):
    c, pos = s["case"], s["pos"].double()
    if s["sections"] is None:
        f = pos[..., None] * s["freqs"]
    else:
        axis = torch.repeat_interleave(torch.tensor(s["sections"], device="cuda"), output_size=s["freqs"].shape[0])
        f = pos[axis].movedim(0, -1) * s["freqs"]
    cos, sin = ((fn(f) * s["amplitude"]).float() for fn in (torch.cos, torch.sin))
    if c["batch"]:  # [B, H, N, d]
        cos, sin = (t.reshape(-1, 1, c["tokens"], t.shape[-1]) for t in (cos, sin))
    else:  # [T, H, d]
        cos, sin = cos[:, None], sin[:, None]
    q = _turn(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    if s["k"] is None:
        return q
    return q, _turn(s["k"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)


def _places(rows, starts, lens, table):
    """Of packed rows: sequence, first of its positions, own position and page."""
    row = torch.arange(rows, device="cuda")
    b = torch.searchsorted(starts[1:].long(), row, right=True)
    start = lens.long()[b] - (starts[1:] - starts[:-1]).long()[b]
    p = start + row - starts.long()[b]
    return b, start, p, table[b, p // PAGE].long()


def _plain_append(s):
    _, start, p, page = _places(s["rows"], s["starts"], s["lens"], s["table"])
    slot = p % PAGE
    older = torch.zeros(s["cache"][0].shape[0], dtype=torch.bool, device="cuda")
    older[page] = p - slot < start
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    head = torch.gather(s["table"].long(), 1, (first // PAGE)[:, None])[:, 0]
    hundred27 = torch.tensor(127.0, device="cuda")
    for codes, scale, x in ((s["cache"][0], s["cache"][1], s["k"].float()), (s["cache"][2], s["cache"][3], s["v"].float())):
        most = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax") / hundred27
        now = torch.where(older[:, None], torch.maximum(scale, most), most)
        ratio = torch.where(older[:, None] & (now > 0), scale / now, torch.ones_like(now))
        codes[head] = (codes[head].float() * ratio[head][:, :, None, None]).round().to(torch.int8)
        by = now[page][:, :, None]
        codes[page, :, slot] = torch.where(by > 0, x / by, torch.zeros_like(x)).round().clamp(-127, 127).to(torch.int8)
        scale[page] = now[page]
    _, _, p, page = _places(s["seen"], s["seen_starts"], s["lens"], s["table"])
    return tuple(c[page, :, p % PAGE].float() * sc[page][:, :, None] for c, sc in (s["cache"][:2], s["cache"][2:]))


def _plain_attn(s):
    c, q = s["case"], s["q"]
    kv, d, batch, widest = c["k_heads"], c["d"], c["batch"], s["widest"]
    group = c["q_heads"] // kv
    table = s["table"].long()

    def dense(codes, scale):
        x = codes[table].float() * scale[table][..., None, None]  # [B, pages, heads, 64, d]
        return x.transpose(1, 2).reshape(batch, kv, -1, d)

    n = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(widest, device="cuda")
    at = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["rows"] - 1)
    rows = q.float()[at].reshape(batch, widest, kv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, kv, widest * group, d)
    x = (rows @ dense(s["cache"][0], s["cache"][1]).transpose(2, 3)).mul_(s["scale"])
    x = x.reshape(batch, kv, widest, group, -1)
    t = torch.arange(x.shape[-1], device="cuda")
    p = (s["lens"].long() - n)[:, None, None] + i[:, None]
    sees = t < s["lens"].long()[:, None, None]
    if c.get("causal", True):
        sees = sees & (t <= p)
    if c["window"] > 0:
        sees = sees & (t > p - c["window"])
    x.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    most = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    x.sub_(most).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(batch, kv, widest * group, -1) @ dense(s["cache"][2], s["cache"][3])).reshape(batch, kv, widest, group, d)
    o, lse = o / total, (most + total.log())[..., 0]
    b = torch.searchsorted(s["starts"][1:].long(), torch.arange(s["rows"], device="cuda"), right=True)
    j = torch.arange(s["rows"], device="cuda") - s["starts"].long()[b]
    return o[b, :, j].reshape(s["rows"], kv * group, d).to(q.dtype), lse[b, :, j].reshape(s["rows"], kv * group)


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "decode": _plain_attn, "chunk": _plain_attn}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_attn, "chunk": _exact_attn}[case["op"]](state)


def _exact_rope(s):
    c, rot = s["case"], s["case"]["rot"]
    out = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y = x.double().clone()
        z = y if c["batch"] else y.transpose(0, 1)  # tokens in front of the channels
        axis = 0
        for i in range(rot // 2):
            if s["sections"] is not None:
                ends = np.cumsum(s["sections"])
                axis = int(np.searchsorted(ends, i, side="right"))
            p = (s["pos"] if s["sections"] is None else s["pos"][axis]).double()
            f = p * s["freqs"][i]
            cos, sin = torch.cos(f) * s["amplitude"], torch.sin(f) * s["amplitude"]
            if c["batch"] and s["sections"] is None:
                cos, sin = cos[:, None], sin[:, None]
            u, w = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            a, b = z[..., u].clone(), z[..., w].clone()
            z[..., u], z[..., w] = a * cos - b * sin, b * cos + a * sin
        out.append(y)
    return out[0] if len(out) == 1 else tuple(out)


def _exact_append(s):
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    starts = s["starts"].cpu().numpy()

    def fl(x):  # one rounding to 32 bits
        return x.astype(np.float32).astype(np.float64)

    result = []
    for codes, scale, x in ((s["cache"][0], s["cache"][1], s["k"]), (s["cache"][2], s["cache"][3], s["v"])):
        parts = []
        for b, length in enumerate(lens):
            length = int(length)
            y = x[int(starts[b]):int(starts[b + 1])].cpu().double().numpy()  # [n, heads, d]
            start = length - y.shape[0]
            for j in range(start // PAGE, -(-length // PAGE)):
                lo, hi = max(start, PAGE * j), min(length, PAGE * j + PAGE)
                new = y[lo - start:hi - start]
                old = lo - PAGE * j
                page = int(table[b, j])
                top = fl(np.abs(new).max((0, 2)) / 127.0)
                before = scale[page].cpu().double().numpy()
                top = np.maximum(top, before) if old else top
                div = np.where(top > 0, top, 1.0)
                if old:
                    was = codes[page, :, :old].cpu().double().numpy()  # [heads, old, d]
                    c = np.rint(fl(was * fl(before / div)[:, None, None]))
                    parts.append(np.transpose(c * top[:, None, None], (1, 0, 2)))
                c = np.clip(np.rint(fl(new / div[None, :, None])), -127, 127)
                parts.append(c * top[None, :, None])
        result.append(np.concatenate(parts))
    return tuple(result)


def _exact_attn(s):
    c, q = s["case"], s["q"].double()
    group, heads = c["q_heads"] // c["k_heads"], c["q_heads"]
    o = torch.zeros(s["rows"], heads, c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], heads), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, first, last) in enumerate(_spans(c)):
        length = int(s["lens"][b])
        t = torch.arange(length, device="cuda")
        page, slot = s["table"][b].long()[t // PAGE], t % PAGE
        first, last = torch.from_numpy(first).cuda(), torch.from_numpy(last).cuda()
        sees = (t >= first[:, None]) & (t <= last[:, None])
        for h in range(c["k_heads"]):
            k, v = (cc[page, h, slot].double() * ss[page, h].double()[:, None] for cc, ss in (s["cache"][:2], s["cache"][2:]))
            for g in range(h * group, (h + 1) * group):
                x = (q[at:at + n, g] @ k.T) * s["scale"]
                x.masked_fill_(~sees, -math.inf)
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                o[at:at + n, g] = torch.exp(x - lse[at:at + n, g][:, None]) @ v
        at += n
    return o, lse
