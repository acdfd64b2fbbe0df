"""Operators over the low-bit KV cache for several tokens of a sequence at once: cases and plain forms.

Four operators, each in a plain form (elementary torch operations) and as the calls that a user makes:

  append  a run of new tokens of each sequence: keys and queries rotated to their positions, keys and
          values moved into the cache (window ring, then 2/3/4-bit codes, contiguous or paged)
  read    tokens of the cache read back as the values they stand for
  chunk   causal attention of each sequence's newest tokens over everything in the cache
  cross   full attention of a run of queries over a cache of another length (an encoder's states)

`own` chooses the side that `run` takes.  Lengths are ragged and follow from the case alone; contents
follow from the seed.
"""

import math

import torch

own = False

GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------- cases ---


def _case(name, op, batch, hq, hkv, d, bits, residual, sink, paged, kv_min, kv_max, q_min, q_max,
          rotary=0, interleaved=False):
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, bits=bits, residual=residual, sink=sink,
             paged=paged, kv_min=kv_min, kv_max=kv_max, q_min=q_min, q_max=q_max, rotary=rotary,
             interleaved=interleaved)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one sequence, its window full: the serving loop's append, where latency counts
        _case("append-token", "append", 1, 32, 8, 128, 4, 128, 0, False, 1000, 1000, 1, 1, 128),
        # drafts of a speculative step, 1 to 8 tokens for each of 16 sequences, paged
        _case("append-draft-b16", "append", 16, 32, 8, 128, 4, 128, 0, True, 1024, 4096, 1, 8, 128),
        # ragged pieces of four prompts, codes of 2 bits, half of each head rotated in adjacent pairs
        _case("append-prompt-int2", "append", 4, 32, 8, 128, 2, 128, 0, False, 300, 9000, 501, 4096, 64, True),
        # the newest tokens of eight sequences read back, heads of 64, 3 bits
        _case("read-recent-int3", "read", 8, 8, 8, 64, 3, 64, 0, False, 200, 1111, 1, 256),
        # a whole 32K layer read back
        _case("read-32k", "read", 1, 32, 8, 128, 4, 128, 0, False, 32768, 32768, 32768, 32768),
        # five drafted tokens checked against 32K tokens
        _case("verify-32k", "chunk", 1, 32, 8, 128, 4, 128, 0, False, 32768, 32768, 5, 5),
        # a batch of drafts, ragged in both lengths, paged
        _case("verify-b16-ragged", "chunk", 16, 32, 8, 128, 4, 128, 0, True, 1024, 8192, 1, 8),
        # pieces of prompts with a head of its own for each query head, an attention sink
        _case("chunk-mha-ragged", "chunk", 4, 40, 40, 128, 4, 96, 32, False, 1024, 4096, 100, 700),
        # a piece of 2048 tokens of a long prompt, 2 bits
        _case("chunk-2048-32k-int2", "chunk", 1, 32, 8, 128, 2, 128, 0, False, 32768, 32768, 2048, 2048),
        # one decoder token for each of 16 encoder states
        _case("cross-token-b16", "cross", 16, 16, 16, 64, 4, 0, 0, False, 200, 1500, 1, 1),
        # whole decoder prompts over encoder states, ragged in both lengths
        _case("cross-prompt-d64", "cross", 8, 16, 16, 64, 4, 0, 0, False, 300, 1500, 7, 448),
        # long queries over long states with shared heads
        _case("cross-16k-gqa", "cross", 2, 32, 8, 128, 4, 0, 0, True, 9999, 16384, 1024, 1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "chunk", "chunk", "cross"])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    gq = rng.choice([1, 1, 2, 3, 4, 4, 8])
    d = rng.choice([32, 64, 64, 128, 128, 128, 256])
    bits = rng.choice([2, 3, 4, 4])
    residual = 0 if op == "cross" else rng.choice([0, 1, 16, 33, 64, 100, 128])
    sink = 0 if op == "cross" else rng.choice([0, 0, 0, 4, 32])
    paged = rng.choice([False, False, True])
    batch = _log_int(rng, 1, 32)
    q_max = _log_int(rng, 1, 2048)
    kv_max = q_max + sink + residual + _log_int(rng, 1, 16384)
    rotary = 0
    interleaved = False
    if op == "append":
        rotary = rng.choice([0, d // 2, d, d])
        interleaved = rng.choice([False, True])
    # no more work than the largest listed case of its kind
    most = 32 * 128 * 2048 * 32768 // 4
    while hkv * gq * max(d, 128) * q_max * kv_max > most:
        q_max, kv_max = max(1, q_max // 2), max(q_max + sink + residual, kv_max // 2)
    while batch > 1 and (batch * hkv * gq * max(d, 128) * q_max * kv_max > most
                         or batch * hkv * d * kv_max > 16 * 8 * 128 * 8192):
        batch = (batch + 1) // 2
    q_min = rng.choice([q_max, max(1, q_max // 3), 1])
    kv_min = rng.choice([kv_max, max(q_max + sink + residual, kv_max // 3)])
    return _case(None, op, batch, hkv * gq, hkv, d, bits, residual, sink, paged, kv_min, kv_max,
                 q_min, q_max, rotary, interleaved)


def _spread(lo, hi, n, shift):
    """n whole numbers of lo..hi, hi the first of them, spread by the golden ratio."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * GOLDEN + shift) % 1.0)) for i in range(n)]


def lengths(case):
    """Tokens in the cache and tokens of the run, for each sequence.  `chunk`: the run is the cache's
    newest tokens; `append`: the cache before the run; `read`: the run is what is read, from the end."""
    b = case["batch"]
    kv = _spread(case["kv_min"], case["kv_max"], b, 0.25)
    q = _spread(case["q_min"], case["q_max"], b, 0.5)
    if case["op"] in ("chunk", "read"):
        q = [min(x, n) for x, n in zip(q, kv)]
    return kv, q


def split(case):
    """(sink, packed, window) tokens of each sequence."""
    kv, _ = lengths(case)
    ns = [min(case["sink"], n) for n in kv]
    nr = [min(case["residual"], n - s) for n, s in zip(kv, ns)]
    return ns, [n - s - r for n, s, r in zip(kv, ns, nr)], nr


def capacity(case):
    cap = max(split(case)[1]) + (case["q_max"] if case["op"] == "append" else 0)
    return max(32, -(-cap // 32) * 32)


def _row_bytes(case):
    """Bytes of one packed token of one KV head, K and V: codes and a (scale, min) pair for 32 values."""
    return 2 * (case["d"] * case["bits"] // 8 + case["d"] // 32 * 4)


def work(case):
    d, hq, hkv, nr = case["d"], case["hq"], case["hkv"], case["residual"]
    kv, q = lengths(case)
    ns, npk, nw = split(case)
    full = 2 * 2 * d  # bytes of K and V of a token of one head in 16 bits
    total = sum(q)
    if case["op"] == "append":
        packed = [max(0, w + t - nr) for w, t in zip(nw, q)]
        old = [min(w, p) for w, p in zip(nw, packed)]  # window tokens read to be packed
        kept = [min(t, nr) for t in q]                 # new tokens that end in the window
        seen = [w + t for w, t in zip(nw, q)]          # what is read back: this run's codes and the window
        b = total * (hkv * full + 4 * hq * d + 4 * case["rotary"])
        b += hkv * (sum(old) * full + sum(packed) * _row_bytes(case) + sum(kept) * full)
        b += hkv * (sum(packed) * _row_bytes(case) + sum(min(w + t, nr) for w, t in zip(nw, q)) * full)
        b += hkv * sum(seen) * full
        return {"bytes": b, "flops": total * (hq + hkv) * case["rotary"] * 3}
    if case["op"] == "read":
        coded = [max(0, min(t - w, p)) for t, w, p in zip(q, nw, npk)]
        plain = [t - c for t, c in zip(q, coded)]
        return {"bytes": hkv * (sum(coded) * _row_bytes(case) + sum(plain) * full + total * full),
                "flops": hkv * sum(coded) * 4 * d}
    if case["op"] == "chunk":
        pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(q, kv))
    else:
        pairs = sum(t * n for t, n in zip(q, kv))
    cache = hkv * (sum(npk) * _row_bytes(case) + (sum(ns) + sum(nw)) * full)
    return {"bytes": cache + total * hq * d * 4, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs ---


def _quantize(x, bits):
    """Groups of 32 along the last dimension: whole codes, scale and min (both rounded to 16 bits)."""
    g = x.float().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    levels = torch.full((1,), float(2 ** bits - 1), device=x.device)
    scale = ((hi - lo) / levels).half()
    s = scale.float()
    code = torch.where(s == 0, 0.0, torch.round((g - lo) / torch.where(s == 0, 1.0, s)))
    return code.clamp(0, 2 ** bits - 1), scale, (lo + 0.0).half()


def _pack(code, bits):
    """Codes [..., groups, 32] as a little-endian bit string, uint8 [..., groups * 4 * bits]."""
    c = code.to(torch.int32).unflatten(-1, (4, 8))  # eight codes: `bits` whole bytes
    at = torch.arange(8, device=code.device, dtype=torch.int32) * bits
    word = (c.to(torch.int64) << at).sum(-1)
    byte = torch.arange(bits, device=code.device) * 8
    return ((word.unsqueeze(-1) >> byte) & 255).to(torch.uint8).flatten(-3)


def _unpack(codes, bits):
    """The inverse: uint8 [..., groups * 4 * bits] -> float [..., groups, 32]."""
    by = codes.unflatten(-1, (-1, 4, bits)).to(torch.int32)
    byte = torch.arange(bits, device=codes.device, dtype=torch.int32) * 8
    word = (by << byte).sum(-1, dtype=torch.int32) if bits < 4 else by[..., 0] | by[..., 1] << 8 | by[..., 2] << 16 | by[..., 3] << 24
    at = torch.arange(8, device=codes.device, dtype=torch.int32) * bits
    return ((word.unsqueeze(-1) >> at) & (2 ** bits - 1)).flatten(-2).float()


def _tokens(gen, shape, d, spread):
    """Normal values; `spread`: a few channels larger, as keys have them."""
    x = torch.randn(*shape, d, generator=gen, device="cuda", dtype=torch.float32)
    if spread:
        x = x * (0.5 + 2.0 * torch.rand(d, generator=gen, device="cuda") ** 6)
    return x.half()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(int(seed))
    B, H, HQ, d, bits, nr, sink = (case[k] for k in ("batch", "hkv", "hq", "d", "bits", "residual", "sink"))
    kv, q = lengths(case)
    ns, npk, nw = split(case)
    cap = capacity(case)
    total, q_max = sum(q), max(q)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [0]
    for t in q:
        cu.append(cu[-1] + t)
    s = dict(case=case, B=B, total=total, q_max=q_max, cap=cap, cu=ints(cu),
             sink_len=ints(ns), packed_len=ints(npk), res_len=ints(nw),
             res_head=ints([(7 * i + 3) % nr if nr and w == nr else 0 for i, w in enumerate(nw)]))
    # the cache's arrays, in the cache's own layout
    for x in ("k", "v"):
        code, scale, lo = _quantize(_tokens(gen, (B, H, cap), d, x == "k"), bits)
        codes = _pack(code, bits)
        params = torch.cat([scale, lo], -1).contiguous().view(torch.int32).squeeze(-1)
        if case["paged"]:
            pages = B * (cap // 32)
            if x == "k":
                s["block_table"] = torch.randperm(pages, generator=gen, device=dev).int().view(B, cap // 32)
            at = s["block_table"].long().flatten()
            pool = lambda t: torch.empty(pages, H, 32, t.shape[-1], dtype=t.dtype, device=dev).index_copy_(  # noqa: E731
                0, at, t.unflatten(2, (-1, 32)).transpose(1, 2).flatten(0, 1))
            codes, params = pool(codes), pool(params)
        s[x + "_codes"], s[x + "_params"] = codes, params
        s[x + "_res"] = _tokens(gen, (B, H, nr), d, x == "k")
        s[x + "_sink"] = _tokens(gen, (B, H, sink), d, x == "k")
    # where each token of the run sits: its sequence and its place in it
    lens = ints(q)
    s["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), lens.long(), output_size=total)
    s["place"] = torch.arange(total, device=dev) - s["cu"].long()[s["seq"]]
    s["lens"] = lens
    if case["op"] == "read":
        s["first"] = ints([n - t for n, t in zip(kv, q)])
    else:
        s["q"] = _tokens(gen, (total, HQ), d, False)
    if case["op"] == "append":
        s["k"], s["v"] = _tokens(gen, (total, H), d, True), _tokens(gen, (total, H), d, False)
        s["first"] = ints([a + b for a, b in zip(ns, npk)])
        if case["rotary"]:
            half = case["rotary"] // 2
            turn = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) * 2 / case["rotary"])
            angle = torch.arange(case["kv_max"] + q_max, device=dev, dtype=torch.float64).unsqueeze(1) * turn
            # cosine and sine of each position, made once as a model's weights are
            s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    if own:
        s["cache"] = _cache(s)
    return s


def _cache(s):
    """The same cache as the framework holds it, with the workspace that a serving program keeps."""
    from bit_quantized_kv_pack_gb300 import kvq

    c = s["case"]
    cache = kvq.KVCache(s["B"], c["hkv"], c["d"], c["bits"], s["cap"], c["residual"], sink=c["sink"],
                        page_size=32 if c["paged"] else 0,
                        num_pages=s["B"] * (s["cap"] // 32) if c["paged"] else 0)
    for name in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "k_sink", "v_sink"):
        getattr(cache, name).copy_(s[name])
    if c["paged"]:
        cache.block_table.copy_(s["block_table"])
    cache.counters.copy_(torch.stack([s["packed_len"], s["res_len"], s["res_head"], s["sink_len"]]))
    s["counters"] = cache.counters.clone()
    if c["op"] in ("chunk", "cross"):
        s["workspace"] = kvq.chunk_workspace_for(cache, c["hq"])
    return cache


# -------------------------------------------------------------- plain forms ---


def _packed_values(s, x):
    """The packed tokens' values [B][H][cap][d] in 32 bits: min + code * scale."""
    codes, params = s[x + "_codes"], s[x + "_params"]
    if s["case"]["paged"]:
        at = s["block_table"].long()
        codes = codes[at].transpose(1, 2).flatten(2, 3)
        params = params[at].transpose(1, 2).flatten(2, 3)
    p = params.unsqueeze(-1).view(torch.float16).float()
    return (p[..., 1:] + _unpack(codes, s["case"]["bits"]) * p[..., :1]).flatten(-2)


def _values(s, x, n):
    """The first n tokens of each sequence in their order, [B][H][n][d] in 32 bits; zeros past its end."""
    c = s["case"]
    nr, sink, cap = c["residual"], c["sink"], s["cap"]
    every = torch.cat([s[x + "_sink"].float(), _packed_values(s, x), s[x + "_res"].float()], 2)
    j = torch.arange(n, device="cuda")
    ns, npk, nw, head = (s[k].long().unsqueeze(1) for k in ("sink_len", "packed_len", "res_len", "res_head"))
    ring = sink + cap + (j - ns - npk + head) % max(nr, 1)
    at = torch.where(j < ns, j, torch.where(j < ns + npk, sink + j - ns, ring))
    live = j < ns + npk + nw
    at = torch.where(live, at, 0)
    got = torch.take_along_dim(every, at[:, None, :, None], 2)
    return torch.where(live[:, None, :, None], got, 0.0)


def _rotated(s, x):
    """x [total][heads][d] rotated to the positions of the run's tokens, rounded once to 16 bits."""
    c = s["case"]
    r = c["rotary"]
    if not r:
        return x
    at = (s["sink_len"] + s["packed_len"] + s["res_len"]).long()[s["seq"]] + s["place"]
    cos, sin = s["rope"][at].unsqueeze(1).unbind(-1)
    f = x[..., :r].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if c["interleaved"] else (f[..., : r // 2], f[..., r // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    f = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([f.half(), x[..., r:]], -1)


def _append(s):
    """The window and the new tokens in order: what no longer fits the window becomes codes."""
    c = s["case"]
    nr = c["residual"]
    n = nr + s["q_max"]
    nw, t = s["res_len"].long(), s["lens"].long()
    packed = (nw + t - nr).clamp(min=0)
    j = torch.arange(n, device="cuda")
    out = {}
    for x, new in (("k", _rotated(s, s["k"])), ("v", s["v"])):
        line = torch.zeros(s["B"], n, c["hkv"], c["d"], dtype=torch.float16, device="cuda")
        if nr:
            ring = (s["res_head"].long().unsqueeze(1) + j[:nr]) % nr
            old = torch.take_along_dim(s[x + "_res"], ring[:, None, :, None], 2).transpose(1, 2)
            line[:, :nr] = torch.where((j[:nr] < nw.unsqueeze(1))[:, :, None, None], old, 0.0)
        line[s["seq"], nw[s["seq"]] + s["place"]] = new
        code, scale, lo = _quantize(line, c["bits"])
        coded = (lo.float() + code * scale.float()).flatten(-2).half()
        line = torch.where((j < packed.unsqueeze(1))[:, :, None, None], coded, line)
        out[x] = line.transpose(1, 2)
    head = (s["res_head"].long() + packed) % nr if nr else s["res_head"].long()
    out["q"] = _rotated(s, s["q"])
    out["counters"] = torch.stack([s["packed_len"].long() + packed, nw + t - packed, head, s["sink_len"].long()]).int()
    return out


def _attend(s, causal):
    c = s["case"]
    n, gq = c["kv_max"], c["hq"] // c["hkv"]
    size = (s["sink_len"] + s["packed_len"] + s["res_len"]).long()
    q = torch.zeros(s["B"], s["q_max"], c["hkv"], gq, c["d"], device="cuda")
    q[s["seq"], s["place"]] = s["q"].float().unflatten(1, (c["hkv"], gq))
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B][H][gq * q_max][d]
    score = (q * (1 / math.sqrt(c["d"]))) @ _values(s, "k", n).transpose(-1, -2)
    seen = size.unsqueeze(1).expand(-1, s["q_max"])
    if causal:
        seen = size.unsqueeze(1) - s["lens"].long().unsqueeze(1) + 1 + torch.arange(s["q_max"], device="cuda")
    hidden = torch.arange(n, device="cuda") >= seen.unsqueeze(-1)  # [B][q_max][n]
    score = score.unflatten(2, (gq, s["q_max"])).masked_fill_(hidden[:, None, None], float("-inf"))
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    score.exp_()
    score /= score.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (score.flatten(2, 3) @ _values(s, "v", n)).unflatten(2, (gq, s["q_max"]))
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["seq"], s["place"]].half()


# --------------------------------------------------------------------- runs ---


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _calls(s, op)
    if op == "append":
        return _append(s)
    if op == "read":
        n, t = s["case"]["kv_max"], s["q_max"]
        j = s["first"].long().unsqueeze(1) + torch.arange(t, device="cuda")
        live = j < (s["first"] + s["lens"]).long().unsqueeze(1)
        at = torch.where(live, j, 0)[:, None, :, None]
        return {x: torch.where(live[:, None, :, None], torch.take_along_dim(_values(s, x, n), at, 2), 0.0).half()
                for x in ("k", "v")}
    return _attend(s, op == "chunk")


def _calls(s, op):
    from bit_quantized_kv_pack_gb300 import kvq

    cache = s["cache"]
    if op == "append":
        # back to the state before the run, as after a rejected draft: the counters and the window
        cache.counters.copy_(s["counters"])
        if s["case"]["residual"]:
            torch._foreach_copy_([cache.k_res, cache.v_res], [s["k_res"], s["v_res"]])
        q = kvq.kvq_append_chunk(cache, s["k"], s["v"], s["cu"], s["q_max"], q=s["q"], rope=s.get("rope"),
                                 interleaved=s["case"]["interleaved"])
        k, v = kvq.kvq_read_tokens(cache, s["first"], s["case"]["residual"] + s["q_max"])
        return {"k": k, "v": v, "q": q, "counters": cache.counters}
    if op == "read":
        k, v = kvq.kvq_read_tokens(cache, s["first"], s["q_max"])
        return {"k": k, "v": v}
    attend = kvq.kvq_chunk_attention if op == "chunk" else kvq.kvq_cross_attention
    return attend(cache, s["q"], s["cu"], s["q_max"], workspace=s["workspace"])


# -------------------------------------------------------------------- exact ---


def _exact_tokens(s, x, b):
    """Sequence b's tokens [H][n][d] in 64 bits, read element by element from the cache's layout."""
    c = s["case"]
    bits, d, H = c["bits"], c["d"], c["hkv"]
    ns, npk, nw, head = (int(s[k][b]) for k in ("sink_len", "packed_len", "res_len", "res_head"))
    t = torch.arange(npk, device="cuda")
    if c["paged"]:
        page = s["block_table"][b].long()[t // 32]
        codes, params = s[x + "_codes"][page, :, t % 32].transpose(0, 1), s[x + "_params"][page, :, t % 32].transpose(0, 1)
    else:
        codes, params = s[x + "_codes"][b, :, :npk], s[x + "_params"][b, :, :npk]
    e = torch.arange(d, device="cuda")
    # element e is the bits [e * bits, e * bits + bits) of its row
    wide = torch.cat([codes, torch.zeros_like(codes[..., :1])], -1).long()
    pair = wide[..., e * bits // 8] + 256 * wide[..., e * bits // 8 + 1]
    code = (pair >> (e * bits % 8)) % 2 ** bits
    p = params.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).double()
    scale, lo = (p[..., i].repeat_interleave(32, -1) for i in (0, 1))
    ring = (head + torch.arange(nw, device="cuda")) % max(c["residual"], 1)
    return torch.cat([s[x + "_sink"][b, :, :ns].double(), lo + code * scale, s[x + "_res"][b][:, ring].double()], 1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kv, q = lengths(case)
    ns, npk, nw = split(case)
    d, H, HQ, nr, bits, B = (case[k] for k in ("d", "hkv", "hq", "residual", "bits", "batch"))
    gq = HQ // H
    at = [0]
    for t in q:
        at.append(at[-1] + t)
    if case["op"] == "read":
        out = {x: torch.zeros(B, H, max(q), d, dtype=torch.float64, device="cuda") for x in "kv"}
        for x in "kv":
            for b in range(B):
                out[x][b, :, : q[b]] = _exact_tokens(s, x, b)[:, kv[b] - q[b]:]
        return out
    if case["op"] == "append":
        n = nr + max(q)
        out = {x: torch.zeros(B, H, n, d, dtype=torch.float64, device="cuda") for x in "kv"}

        def turned(x, b):
            x, r = x.double(), case["rotary"]
            if not r:
                return x
            i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
            pos = torch.arange(kv[b], kv[b] + q[b], device="cuda", dtype=torch.float64)
            angle = (pos[:, None] * torch.exp(-math.log(10000.0) * 2 * i / r))[:, None]
            first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            y = x.clone()
            y[..., first] = x[..., first] * angle.cos() - x[..., second] * angle.sin()
            y[..., second] = x[..., second] * angle.cos() + x[..., first] * angle.sin()
            return y

        counters, rotated = [], []
        for b in range(B):
            mine = slice(at[b], at[b + 1])
            rotated.append(turned(s["q"][mine], b))
            p = max(0, nw[b] + q[b] - nr)
            ring = [(int(s["res_head"][b]) + i) % nr for i in range(nw[b])]
            for x in "kv":
                new = s[x][mine].double() if x == "v" else turned(s["k"][mine], b)
                line = torch.cat([s[x + "_res"][b][:, ring].double(), new.transpose(0, 1)], 1)
                g = line[:, :p].half().double().unflatten(-1, (-1, 32))
                lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
                scale = ((hi - lo) / (2 ** bits - 1)).half().double()
                code = torch.where(scale > 0, ((g - lo) / scale.clamp(min=1e-30)).round().clamp(0, 2 ** bits - 1), 0.0)
                out[x][b, :, :p] = (lo + code * scale).flatten(-2)
                out[x][b, :, p:nw[b] + q[b]] = line[:, p:]
            counters.append([npk[b] + p, nw[b] + q[b] - p, (int(s["res_head"][b]) + p) % nr if nr else 0, ns[b]])
        out["q"] = torch.cat(rotated)
        out["counters"] = torch.tensor(counters, dtype=torch.int32).t().contiguous()
        return out
    out = torch.empty(at[-1], HQ, d, dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = _exact_tokens(s, "k", b), _exact_tokens(s, "v", b)
        for h in range(HQ):
            for lo in range(0, q[b], 1024):
                rows = torch.arange(lo, min(q[b], lo + 1024), device="cuda")
                x = s["q"][at[b] + rows, h].double() @ k[h // gq].T / math.sqrt(d)
                if case["op"] == "chunk":
                    x.masked_fill_(torch.arange(kv[b], device="cuda") > (kv[b] - q[b] + rows)[:, None], float("-inf"))
                out[at[b] + rows, h] = torch.softmax(x, -1) @ v[h // gq]
    return out
