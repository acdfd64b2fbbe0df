"""Operators of a generation with beams from a prompt of text and images: cases and plain forms.

Four operators around the low-bit KV cache, each in a plain form (elementary torch operations) and as the
calls that a user makes:

  rotate   rotary positions with several axes (time, height, width) of queries and keys, before attention
  prompt   causal attention over whole prompts in full precision, sequences of different lengths packed
           one after the other, shared key/value heads: what runs before the cache is packed
  select   beam search's selection over beams and vocabulary
  reorder  the cache's sequences follow the selected beams: codes, parameters, window and sink move, or,
           with shared pages, the last page, the window and the block table alone

`own` chooses the side that `run` takes.  Lengths and positions follow from the case alone; contents
follow from the seed.
"""

import math

import torch

own = False

GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------- cases ---


def _rotate(name, batch, n_min, n_max, hq, hkv, d, rotary, axes, mixed, interleaved):
    """mixed: the axes take the pairs in turn; otherwise each has a run of them."""
    return _named(name, op="rotate", batch=batch, n_min=n_min, n_max=n_max, hq=hq, hkv=hkv, d=d, rotary=rotary,
                  axes=axes, mixed=mixed, interleaved=interleaved)


def _prompt(name, batch, n_min, n_max, hq, hkv, d, f32=False):
    return _named(name, op="prompt", batch=batch, n_min=n_min, n_max=n_max, hq=hq, hkv=hkv, d=d, f32=f32)


def _select(name, batch, beams, vocab, n, f32, first=False, ended=False, banned=0):
    """first: the first step, all beams but one of each batch entry without a score; ended: some beams are
    complete; banned: tokens whose logit is -inf."""
    return _named(name, op="select", batch=batch, beams=beams, vocab=vocab, n=n, f32=f32, first=first,
                  ended=ended, banned=banned)


def _reorder(name, batch, hkv, d, bits, residual, sink, kv_min, kv_max, paged=False, share=False):
    return _named(name, op="reorder", batch=batch, hkv=hkv, d=d, bits=bits, residual=residual, sink=sink,
                  n_min=kv_min, n_max=kv_max, paged=paged, share=share)


def _named(name, **c):
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of each of 16 sequences, before the decode step: latency counts
        _rotate("rotate-token-b16", 16, 1, 1, 32, 8, 128, 128, 3, False, False),
        # packed prompts of text and images, three axes in runs of pairs
        _rotate("rotate-image-prompts", 6, 1000, 9001, 32, 8, 128, 128, 3, False, False),
        # patches of images by row and column, adjacent pairs, heads of 64
        _rotate("rotate-patches-d64", 5, 700, 4100, 16, 16, 64, 64, 2, True, True),
        # a chat turn
        _prompt("prompt-77", 1, 77, 77, 32, 8, 128),
        # a batch of prompts of a server, ragged
        _prompt("prompt-b16-ragged", 16, 17, 2048, 32, 8, 128),
        # heads of 64, each query head with keys of its own, fp32 output
        _prompt("prompt-mha-d64", 8, 100, 1500, 16, 16, 64, True),
        # one long prompt
        _prompt("prompt-16k", 1, 16384, 16384, 32, 8, 128),
        # first step of four beams over 32000 tokens, half precision logits
        _select("select-4x32000-first", 1, 4, 32000, 4, False, first=True),
        # an odd vocabulary, complete beams and banned tokens
        _select("select-3x5x50257", 3, 5, 50257, 10, False, ended=True, banned=300),
        # a batch of beams over a large vocabulary, fp32 logits
        _select("select-16x8x128256", 16, 8, 128256, 16, True),
        # four beams of 32K tokens change places, contiguous cache
        _reorder("reorder-4x32k", 4, 8, 128, 4, 128, 0, 32700, 32768),
        # 32 sequences of a paged cache with an attention sink, full pages shared
        _reorder("reorder-shared-b32", 32, 8, 128, 2, 128, 32, 1000, 8000, paged=True, share=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "select", "reorder"])
    if op == "select":
        beams = _log_int(rng, 1, 16)
        vocab = _log_int(rng, 1000, 200000)
        batch = _log_int(rng, 1, 32)
        while batch > 1 and batch * beams * vocab > 16 * 8 * 128256:
            batch = (batch + 1) // 2
        n = rng.choice([beams, beams, min(32, 2 * beams)])
        ended = rng.choice([False, False, True])
        return _select(None, batch, beams, vocab, n, rng.choice([False, True]),
                       first=not ended and rng.choice([False, False, True]), ended=ended,
                       banned=rng.choice([0, 0, 7, vocab // 3]))
    d = rng.choice([32, 64, 64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    gq = rng.choice([1, 1, 2, 3, 4, 4, 8])
    batch = _log_int(rng, 1, 32)
    if op == "rotate":
        n_max = _log_int(rng, 1, 16384)
        while batch > 1 and batch * n_max * hkv * (gq + 1) * d > 6 * 9001 * 40 * 128:
            batch = (batch + 1) // 2
        while n_max * hkv * (gq + 1) * d > 6 * 9001 * 40 * 128:
            n_max //= 2
        return _rotate(None, batch, rng.choice([n_max, max(1, n_max // 4)]), n_max, hkv * gq, hkv, d,
                       rng.choice([d, d, d // 2]), rng.choice([1, 2, 3, 3, 4]), rng.choice([False, True]),
                       rng.choice([False, True]))
    if op == "prompt":
        n_max = _log_int(rng, 1, 16384)
        most = 32 * 128 * 16384 * 16384
        while hkv * gq * max(d, 128) * n_max * n_max > most:
            n_max = n_max * 3 // 4
        while batch > 1 and (batch * hkv * gq * max(d, 128) * n_max * n_max > most
                             or batch * n_max * hkv * gq * d > 2 * 32 * 128 * 16384):
            batch = (batch + 1) // 2
        return _prompt(None, batch, rng.choice([n_max, max(1, n_max // 3), 1]), n_max, hkv * gq, hkv, d,
                       rng.choice([False, False, True]))
    n_max = _log_int(rng, 40, 32768)
    while batch > 1 and batch * hkv * d * n_max > 4 * 8 * 128 * 32768:
        batch = (batch + 1) // 2
    while hkv * d * n_max > 4 * 8 * 128 * 32768:
        n_max //= 2
    paged = rng.choice([False, True])
    return _reorder(None, batch, hkv, d, rng.choice([2, 3, 4, 4]), rng.choice([0, 1, 33, 128, 128]),
                    rng.choice([0, 0, 4, 32]), rng.choice([n_max, max(1, n_max // 3)]), n_max, paged,
                    paged and rng.choice([False, True]))


def lengths(case):
    """Tokens of each sequence, the longest first, spread by the golden ratio."""
    lo, hi = case["n_min"], case["n_max"]
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * GOLDEN + 0.25) % 1.0)) for i in range(case["batch"])]


def split(case):
    """(sink, packed, window) tokens of each sequence of a cache."""
    out = []
    for n in lengths(case):
        s = min(case["sink"], n)
        w = min(case["residual"], n - s)
        out.append((s, n - s - w, w))
    return out


def capacity(case):
    return max(32, -(-max(p for _, p, _ in split(case)) // 32) * 32 + 32)


def sources(case):
    """The source sequence of each sequence: beams of four change places, some are lost, some doubled."""
    b = case["batch"]
    return [min(b - 1, i // 4 * 4 + (0, 0, 3, 2)[i % 4]) for i in range(b)]


def pair_axes(case):
    """The axis of each pair of a head."""
    n, axes = case["rotary"] // 2, case["axes"]
    if case["mixed"]:
        return [i % axes for i in range(n)]
    ends = {1: [n], 2: [n // 2, n], 3: [n // 4, n // 4 + 3 * n // 8, n],
            4: [n // 4, n // 2, 3 * n // 4, n]}[axes]
    return [next(a for a, e in enumerate(ends) if i < e) for i in range(n)]


def positions(case):
    """Positions of the packed tokens on each axis, int64 [axes][total]: runs of text, on which all axes
    advance together, and images, whose patches differ in frame, row and column."""
    axes, parts = case["axes"], []
    for b, n in enumerate(lengths(case)):
        if n == 1:  # a new token some way into its sequence
            parts.append(torch.full((axes, 1), 37 + 811 * b, dtype=torch.int64))
            continue
        at, left, k = 0, n, 0
        while left > 0:
            k += 1
            text = min(left, 5 + (37 * k + 11 * b) % 60)
            parts.append((at + torch.arange(text)).expand(axes, text))
            at, left = at + text, left - text
            rows, cols = 8 + (13 * k + b) % 40, 8 + (29 * k + 3 * b) % 40
            i = torch.arange(min(left, rows * cols * (1 + k % 2)))
            grid = [i // (rows * cols), i // cols % rows, i % cols, i * 0]
            parts.append(at + torch.stack((grid if axes > 2 else grid[1:])[:axes]))
            at, left = at + max(rows, cols), left - len(i)
    return torch.cat(parts, 1)


def _row_bytes(case):
    """Bytes of one packed token of one KV head, K and V: codes and a (scale, min) pair for 32 values."""
    return 2 * (case["d"] * case["bits"] // 8 + case["d"] // 32 * 4)


def work(case):
    op = case["op"]
    if op == "select":
        rows, n = case["batch"] * case["beams"], case["batch"] * case["n"]
        return {"bytes": rows * (case["vocab"] * (4 if case["f32"] else 2) + 4) + 12 * n,
                "flops": 4 * rows * case["vocab"]}
    if op == "reorder":
        full = 2 * 2 * case["d"]
        b = 0
        for i in sources(case):
            s, p, w = split(case)[i]
            b += case["hkv"] * ((p % 32 if case["share"] else p) * _row_bytes(case) + (s + w) * full) + 16
            b += p // 32 * 4 if case["share"] else 0
        return {"bytes": 2 * b, "flops": 0}
    total, d, hq, hkv = sum(lengths(case)), case["d"], case["hq"], case["hkv"]
    if op == "rotate":
        return {"bytes": total * (hq + hkv) * d * 4 + total * 4 * case["axes"]
                + sum(8 * pair_axes(case).count(a) * len(p.unique()) for a, p in enumerate(positions(case))),
                "flops": 3 * total * (hq + hkv) * case["rotary"]}
    return {"bytes": total * d * (2 * hq + 4 * hkv + hq * (4 if case["f32"] else 2)),
            "flops": sum(2 * d * hq * n * (n + 1) for n in lengths(case))}


# ------------------------------------------------------------------ inputs ---


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _projected(case, gen):
    """Queries, keys and values as views of a fused projection's output [total][(Hq + 2 Hkv) d]."""
    d, hq, hkv, total = case["d"], case["hq"], case["hkv"], sum(lengths(case))
    x = torch.randn(total, hq + 2 * hkv, d, generator=gen, device="cuda", dtype=torch.float32)
    # a few channels of the keys are larger
    x[:, hq:hq + hkv] *= 0.5 + 2.0 * torch.rand(d, generator=gen, device="cuda") ** 6
    return x.half().split([hq, hkv, hkv], 1)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "select":
        _prepare_select(s, case, gen)
    elif case["op"] == "reorder":
        _prepare_reorder(s, case, gen)
    else:
        s["q"], s["k"], s["v"] = _projected(case, gen)
        cu = [0]
        for n in lengths(case):
            cu.append(cu[-1] + n)
        s["cu"], s["ends"] = _ints(cu), cu
    if case["op"] == "rotate":
        pos = positions(case)
        half = case["rotary"] // 2
        turn = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) * 2 / case["rotary"])
        angle = torch.arange(int(pos.max()) + 1, device="cuda", dtype=torch.float64).unsqueeze(1) * turn
        # cosine and sine of each position, made once as a model's weights are
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
        s["positions"] = pos.int().cuda()
        s["pair_axis"] = pair_axes(case)
        s["out"] = [torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"])]
    if case["op"] == "prompt":
        s["out"] = torch.empty(s["q"].shape, dtype=torch.float32 if case["f32"] else torch.float16, device="cuda")
    return s


def _prepare_select(s, case, gen):
    B, W, V, n = case["batch"], case["beams"], case["vocab"], case["n"]
    x = torch.randn(B, W, V, generator=gen, device="cuda") * 2.5
    x += torch.rand(B, W, 1, generator=gen, device="cuda") * 4 - 2
    if case["banned"]:
        x[:, :, torch.randperm(V, generator=gen, device="cuda")[:case["banned"]]] = -math.inf
    s["logits"] = x if case["f32"] else x.half()
    s["scores"] = -20.0 * torch.rand(B, W, generator=gen, device="cuda")
    if case["first"]:
        s["scores"][:, 0] = 0.0
        s["scores"][:, 1:] = -math.inf
    s["end"] = V // 2
    s["ended"] = None
    if case["ended"]:
        s["ended"] = (torch.rand(B, W, generator=gen, device="cuda") < 0.3).to(torch.uint8)
    s["out"] = [torch.empty(B, n, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
    if own:
        from bit_quantized_kv_pack_gb300 import kvq

        s["workspace"] = kvq.beam_workspace_for(B, W, V, n)


ARRAYS = ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "k_sink", "v_sink", "counters")


def _prepare_reorder(s, case, gen):
    B, H, d, bits, nr, sink = (case[k] for k in ("batch", "hkv", "d", "bits", "residual", "sink"))
    cap = capacity(case)
    own_pages = B * cap // 32
    pages = own_pages * (2 if case["share"] else 1)
    rows = (pages, H, 32) if case["paged"] else (B, H, cap)
    src = {}
    for x in "kv":
        src[x + "_codes"] = torch.randint(0, 256, (*rows, d * bits // 8), generator=gen, device="cuda", dtype=torch.uint8)
        p = torch.randn(*rows, d // 32, 2, generator=gen, device="cuda").half()
        src[x + "_params"] = p.view(torch.int32).squeeze(-1)
        src[x + "_res"] = torch.randn(B, H, nr, d, generator=gen, device="cuda").half()
        src[x + "_sink"] = torch.randn(B, H, sink, d, generator=gen, device="cuda").half()
    parts = split(case)
    src["counters"] = _ints([[p for _, p, _ in parts], [w for _, _, w in parts],
                             [(7 * i + 3) % nr if nr and parts[i][2] == nr else 0 for i in range(B)],
                             [a for a, _, _ in parts]])
    dst = {k: src[k] if case["share"] and k[2:] in ("codes", "params") else torch.zeros_like(src[k]) for k in ARRAYS}
    if case["paged"]:
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        src["block_table"] = order[:own_pages].view(B, cap // 32)
        dst["block_table"] = order[-own_pages:].view(B, cap // 32).clone()
    s["src"], s["dst"], s["index"] = src, dst, _ints(sources(case))
    if own:
        from bit_quantized_kv_pack_gb300 import kvq

        a = kvq.KVCache(B, H, d, bits, cap, nr, sink=sink, page_size=32 if case["paged"] else 0,
                        num_pages=pages if case["paged"] else 0)
        b = a.twin(share_pages=case["share"])
        for cache, t in ((a, src), (b, dst)):
            for k in t:
                getattr(cache, k).copy_(t[k])
        s["caches"] = (a, b)


# -------------------------------------------------------------- plain forms ---


def _rotated(s, x):
    """x [total][heads][d] rotated, rounded once to 16 bits."""
    c = s["case"]
    r = c["rotary"]
    axis = torch.tensor(s["pair_axis"], device="cuda")
    at = s["positions"].long()[axis].t()  # [total][pairs]: the table's row of each pair
    cs = torch.take_along_dim(s["rope"], at.unsqueeze(-1), 0).unsqueeze(1)
    cos, sin = cs[..., 0], cs[..., 1]
    f = x[..., :r].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if c["interleaved"] else (f[..., : r // 2], f[..., r // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    f = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([f.half(), x[..., r:]], -1)


def _attended(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    gq = hq // hkv
    out = s["out"]
    for lo, hi in zip(s["ends"], s["ends"][1:]):
        n = hi - lo
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1)
        for h in range(hkv):
            q = s["q"][lo:hi, h * gq:(h + 1) * gq].transpose(0, 1).float() * (1 / math.sqrt(d))
            score = q @ s["k"][lo:hi, h].float().t()  # [gq][n][n]
            score.masked_fill_(later, -math.inf)
            score -= score.amax(-1, keepdim=True)
            score.exp_()
            score /= score.sum(-1, keepdim=True)
            out[lo:hi, h * gq:(h + 1) * gq] = (score @ s["v"][lo:hi, h].float()).transpose(0, 1)
    return out


def _selected(s):
    """The n largest scores of each batch entry over beams and tokens, equal ones in order."""
    c = s["case"]
    B, W, V, n = c["batch"], c["beams"], c["vocab"], c["n"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    norm = top + (x - top).exp().sum(-1, keepdim=True).log()
    base = s["scores"].double().unsqueeze(-1)
    score = base + (x - norm)
    if s["ended"] is not None:
        # a complete beam stays as it is, with the end token
        kept = torch.full_like(score, -math.inf)
        kept[..., s["end"]] = base.squeeze(-1)
        score = torch.where(s["ended"].bool().unsqueeze(-1), kept, score)
    score, at = score.flatten(1).sort(dim=1, descending=True, stable=True)
    score, at = score[:, :n], at[:, :n]
    first = torch.arange(B, device="cuda").unsqueeze(1) * W
    return {"parent": (first + at // V).int(), "token": (at % V).int(), "score": score.float()}


def _moved(s):
    """Live entries of each destination sequence from its source, in place in the destination's arrays."""
    c, src, dst = s["case"], s["src"], s["dst"]
    at = s["index"].long()
    packed, window, head, _ = src["counters"].long()[:, at].unsqueeze(-1)
    cap = capacity(c)
    j = torch.arange(cap, device="cuda")
    live = j < packed
    for x in "kv":
        for name in (x + "_codes", x + "_params"):
            if c["paged"]:
                got = src[name][src["block_table"].long()[at]]  # [B][cap / 32][H][32][...]
                rows = live.unflatten(1, (-1, 32))
                if c["share"]:
                    rows = rows & (j >= packed // 32 * 32).unflatten(1, (-1, 32))
                b, page, r = rows.nonzero(as_tuple=True)
                dst[name][dst["block_table"].long()[b, page], :, r] = got[b, page, :, r]
            else:
                dst[name].copy_(torch.where(live[:, None, :, None], src[name][at], dst[name]))
        if c["residual"]:
            i = torch.arange(c["residual"], device="cuda")
            there = (i - head) % c["residual"] < window
            dst[x + "_res"].copy_(torch.where(there[:, None, :, None], src[x + "_res"][at], dst[x + "_res"]))
        if c["sink"]:
            i = torch.arange(c["sink"], device="cuda")
            there = i < src["counters"][3].long()[at].unsqueeze(1)
            dst[x + "_sink"].copy_(torch.where(there[:, None, :, None], src[x + "_sink"][at], dst[x + "_sink"]))
    dst["counters"].copy_(src["counters"][:, at])
    if c["share"]:
        full = torch.arange(cap // 32, device="cuda") < packed // 32
        dst["block_table"].copy_(torch.where(full, src["block_table"][at], dst["block_table"]))
    return _whole(dst)


def _whole(t):
    """A cache's arrays as outputs.  Codes and parameters move as they are and have to be equal bit for
    bit: they are returned as whole words."""
    words = lambda x: x.view(torch.int32) if x.dtype == torch.uint8 else x  # noqa: E731
    return {k: words(t[k]) for k in (*ARRAYS, "block_table") if k in t and t[k].numel()}


# --------------------------------------------------------------------- runs ---


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _calls(s, op)
    if op == "rotate":
        return {"q": _rotated(s, s["q"]), "k": _rotated(s, s["k"])}
    return _attended(s) if op == "prompt" else _selected(s) if op == "select" else _moved(s)


def _calls(s, op):
    from bit_quantized_kv_pack_gb300 import kvq

    if op == "rotate":
        q, k = kvq.kvq_rotate(s["q"], s["k"], s["rope"], s["positions"], pair_axis=s["pair_axis"],
                              interleaved=s["case"]["interleaved"], q_out=s["out"][0], k_out=s["out"][1])
        return {"q": q, "k": k}
    if op == "prompt":
        return kvq.kvq_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["case"]["n_max"], out=s["out"])
    if op == "select":
        parent, token, score = kvq.kvq_beam_select(s["logits"], s["scores"], s["case"]["n"], finished=s["ended"],
                                                   end_token=s["end"], out=s["out"], workspace=s["workspace"])
        return {"parent": parent, "token": token, "score": score}
    src, dst = s["caches"]
    kvq.kvq_reorder(dst, src, s["index"], share_pages=s["case"]["share"])
    names = (*ARRAYS, "block_table") if s["case"]["paged"] else ARRAYS
    return _whole({k: getattr(dst, k) for k in names})


# -------------------------------------------------------------------- exact ---


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rotate": _exact_rotate, "prompt": _exact_prompt, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](case, s)


def _exact_rotate(case, s):
    r, inter = case["rotary"], case["interleaved"]
    pos = positions(case).cuda().double()
    out = {}
    for x in "qk":
        v = s[x].double()
        y = v.clone()
        for i, axis in enumerate(pair_axes(case)):
            angle = (pos[axis] * math.exp(-math.log(10000.0) * 2 * i / r)).unsqueeze(1)
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
            y[..., a] = v[..., a] * angle.cos() - v[..., b] * angle.sin()
            y[..., b] = v[..., a] * angle.sin() + v[..., b] * angle.cos()
        out[x] = y
    return out


def _exact_prompt(case, s):
    d, gq = case["d"], case["hq"] // case["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths(case)):
        at = int(s["cu"][b])
        for h in range(case["hq"]):
            q, k, v = (s[x][at:at + n, h // (gq if x != "q" else 1)].double() for x in "qkv")
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)  # rows lo .. hi - 1 see the first hi tokens at most
                x = q[lo:hi] @ k[:hi].t() * d ** -0.5
                x[:, lo:].masked_fill_(torch.ones(hi - lo, hi - lo, device="cuda").triu(1).bool(), -math.inf)
                out[at + lo:at + hi, h] = torch.softmax(x, -1) @ v[:hi]
    return out


def _exact_select(case, s):
    B, W, V, n = case["batch"], case["beams"], case["vocab"], case["n"]
    parent, token, score = [], [], []
    for b in range(B):
        rows = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        for w in range(W):
            if s["ended"] is not None and s["ended"][b, w]:
                rows[w] = -math.inf
                rows[w, s["end"]] = s["scores"][b, w].double()
        left = rows.flatten()
        for _ in range(n):
            best = torch.where(left.isnan(), -math.inf, left).max()
            # the first place that holds it; a place that was taken holds NaN
            i = int((left == best).nonzero()[0])
            parent.append(b * W + i // V), token.append(i % V), score.append(float(best))
            left[i] = math.nan
    shape = lambda x, t: torch.tensor(x, dtype=t, device="cuda").view(B, n)  # noqa: E731
    return {"parent": shape(parent, torch.int32), "token": shape(token, torch.int32), "score": shape(score, torch.float64)}


def _exact_reorder(case, s):
    src, dst = s["src"], {k: v.clone() for k, v in s["dst"].items()}
    if case["share"]:
        for k in ARRAYS[:4]:
            dst[k] = src[k].clone()
    nr = max(case["residual"], 1)
    for i, a in enumerate(sources(case)):
        ns, npk, nw = split(case)[a]
        ring = [(int(src["counters"][2, a]) + j) % nr for j in range(nw)]
        for x in "kv":
            for name in (x + "_codes", x + "_params"):
                if not case["paged"]:
                    dst[name][i, :, :npk] = src[name][a, :, :npk]
                    continue
                for p in range(npk // 32 if case["share"] else 0, -(-npk // 32)):
                    rows = min(32, npk - 32 * p)
                    to, of = int(dst["block_table"][i, p]), int(src["block_table"][a, p])
                    dst[name][to, :, :rows] = src[name][of, :, :rows]
            dst[x + "_res"][i][:, ring] = src[x + "_res"][a][:, ring]
            dst[x + "_sink"][i, :, :ns] = src[x + "_sink"][a, :, :ns]
        dst["counters"][:, i] = src["counters"][:, a]
        if case["share"]:
            dst["block_table"][i, :npk // 32] = src["block_table"][a, :npk // 32]
    return _whole(dst)
