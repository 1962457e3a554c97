"""The operators of a layer whose KV cache is held in 4 bits, as measured workloads.

Four operators: appending a projection's keys and values to the paged 4-bit
cache with the position rotation applied on the way ("append"), reading cached
rows back as bf16 ("read"), attention of one query token per request over the
cache ("decode") and attention of prompt tokens over bf16 rows ("prompt").
Each in its plain form (elementary torch operations) and, where `own` is true,
as calls of this repository's library.

A block of one (page, KV head) holds 16 tokens of head size d, W = d / 32:
  [0, 8 d)      K codes: token t's d / 2 bytes at t d / 2; channel
                32 w + 8 u + n (u < 4, n < 8) is nibble n of 32-bit word
                W u + w of the row (nibble 0 = lowest 4 bits);
  [8 d, 16 d)   V codes: channel 32 w + 4 u + n (u < 8, n < 4) of token t is
                nibble 4 (t % 2) + n of 32-bit word (8 (t / 2) + u) W + w;
  [16 d, ...)   token t's K (scale, zero) fp16 pairs, then its V pairs.
"""
import math

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------- the cases

def _case(name, op, batch, lo, hi, n_q, n_kv, d, gk, gv, past=0, rot=0, interleaved=False, theta=1e6, cap=0.0, window=0,
          slopes=False, prefix=0, causal=True):
    c = dict(name=name, op=op, batch=batch, lo=lo, hi=hi, n_q=n_q, n_kv=n_kv, d=d, gk=gk, gv=gv, past=past, rot=rot,
             interleaved=interleaved, theta=theta, cap=cap, window=window, slopes=slopes, prefix=prefix, causal=causal)
    if not name:
        del c["name"]
    return c


def listed():
    return [
        # one new token of one request, deep in its context: what a decode step adds; latency is all
        _case("append-1-token", "append", 1, 1, 1, 32, 8, 128, 128, 128, past=99_999, rot=128),
        # the new tokens of a serving batch of odd size, GQA 8, small groups, rotation of half of each head
        _case("append-61-tokens", "append", 61, 1, 1, 64, 8, 128, 32, 64, past=20_000, rot=64, interleaved=True, theta=1e4),
        # whole prompts of different lengths, 32k tokens together: prefill
        _case("append-prompts", "append", 5, 2_113, 12_001, 32, 8, 128, 64, 64, rot=128),
        # a short shared prefix read back, small heads
        _case("read-short", "read", 3, 97, 501, 16, 4, 64, 64, 32),
        # a long cached prefix read back, so that a prompt can go on from it
        _case("read-prefix", "read", 1, 65_521, 65_521, 32, 8, 128, 128, 128),
        # single tokens: a chat's short context, one request
        _case("decode-1x777", "decode", 1, 777, 777, 32, 8, 128, 128, 128),
        # one request of 100k tokens
        _case("decode-1x100k", "decode", 1, 100_000, 100_000, 32, 8, 128, 128, 128),
        # a ragged batch, GQA 8, small groups, capped scores
        _case("decode-28-ragged-cap", "decode", 28, 2_000, 32_000, 64, 8, 128, 64, 32, cap=50.0),
        # small heads, a group of five, a bias by distance within a window
        _case("decode-16-bias-window", "decode", 16, 301, 9_001, 40, 8, 64, 32, 64, window=4_096, slopes=True),
        # a few new tokens behind a long context (a chat turn after a cached document)
        _case("prompt-24-on-32k", "prompt", 1, 24, 24, 32, 8, 128, 128, 128, past=32_000),
        # packed documents of odd lengths, a bidirectional prefix, capped scores, a group of three
        _case("prompt-ragged-prefix-cap", "prompt", 6, 65, 1_501, 24, 8, 64, 64, 64, cap=30.0, prefix=64),
        # one long prompt
        _case("prompt-8k", "prompt", 1, 8_192, 8_192, 32, 8, 128, 128, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "prompt"])
    d = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    while n_q > 64:
        n_q -= n_kv
    gk, gv = (rng.choice([g for g in (32, 64, 128) if g <= d]) for _ in range(2))
    kw = {}
    if op in ("append", "read"):
        n = _log_int(rng, 1, 29_000 * 32 // max(n_q, 32))
        batch = min(n, _log_int(rng, 1, 200))
        hi = max(1, n // batch)
        kw = dict(rot=rng.choice([0, 16, d // 2, d]), interleaved=rng.random() < 0.5, theta=rng.choice([1e4, 1e6]),
                  past=rng.choice([0, _log_int(rng, 1, 100_000)])) if op == "append" else {}
        return _case("", op, batch, max(1, hi - rng.randrange(0, hi)), hi, n_q, n_kv, d, gk, gv, **kw)
    mods = dict(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, _log_int(rng, 16, 8_000)]),
                slopes=rng.random() < 0.3)
    if op == "decode":
        total = _log_int(rng, 100, 300_000)     # tokens of all requests
        batch = min(total, _log_int(rng, 1, 128))
        hi = max(1, total // batch)
        return _case("", op, batch, max(1, hi // rng.choice([1, 2, 7])), hi, n_q, n_kv, d, gk, gv, **mods)
    total = _log_int(rng, 20, 5_500)            # new tokens of all requests
    batch = min(total, _log_int(rng, 1, 24))
    hi = max(1, total // batch)
    past = rng.choice([0, _log_int(rng, 1, 32_000)]) if hi <= 300 else 0
    past = max(0, min(past, 2 ** 30 // (total * n_q) - hi))
    causal = rng.random() < 0.8
    return _case("", op, batch, max(1, hi // rng.choice([1, 3])), hi, n_q, n_kv, d, gk, gv, past=past, causal=causal,
                 prefix=rng.choice([0, hi // 3]) if causal else 0, **mods)


def _lengths(case):
    """New tokens of each request: from hi down to lo in equal ratios, the longest ones spread over the batch."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    if b == 1 or lo == hi:
        return [hi] * b
    sizes = [int(round(hi * (lo / hi) ** (i / (b - 1)))) for i in range(b)]
    return sizes[0::2] + sizes[1::2]


def _contexts(case):
    """Tokens of each request in all: the new ones and those before them, which differ a little by request."""
    return [n + (max(1, case["past"] - 37 * i) if case["past"] else 0) for i, n in enumerate(_lengths(case))]


def _packed(case):
    """Bytes of one token of one KV head in the cache, K and V together."""
    d = case["d"]
    return d + 4 * (d // case["gk"] + d // case["gv"])


def _visible(case):
    """(query, key) pairs that the mask leaves, over the batch."""
    total = 0
    for n, ctx in zip(_lengths(case), _contexts(case)):
        i = torch.arange(ctx - n, ctx, dtype=torch.int64)
        last = i + 1 if case["causal"] else torch.full_like(i, ctx)
        first = (i - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(i)
        seen = (last - first).clamp(min=0)
        if case["prefix"]:
            pre = min(case["prefix"], ctx)
            seen = torch.clamp(last, min=pre) - torch.where(first <= pre, torch.zeros_like(first), first - pre)
        total += int(seen.sum())
    return total


def work(case):
    n, d, n_q, n_kv = sum(_lengths(case)), case["d"], case["n_q"], case["n_kv"]
    if case["op"] == "append":      # the rows in, the rotated ones out, the codes out, and the cached rows read back
        rows = 2 * d * n * (2 * n_q + 2 * n_kv + n_kv)
        cache = n * n_kv * (2 * _packed(case) + 4 * d)
        return {"bytes": rows + cache + 4 * n * case["rot"], "flops": 3.0 * n * (n_q + n_kv) * case["rot"] + 12.0 * n * n_kv * d}
    if case["op"] == "read":
        return {"bytes": n * n_kv * (_packed(case) + 4 * d), "flops": 4.0 * n * n_kv * d}
    if case["op"] == "decode":
        seen = sum(min(x, case["window"] or x) for x in _lengths(case))
        return {"bytes": seen * n_kv * _packed(case) + 4 * d * n_q * case["batch"], "flops": 4.0 * seen * n_q * d}
    ctx = sum(_contexts(case))
    return {"bytes": 2 * d * (2 * n * n_q + 2 * ctx * n_kv) + 4 * n * n_q, "flops": 4.0 * _visible(case) * n_q * d}


# ------------------------------------------------------------------ the inputs

def _rows(g, n, heads, d, outliers):
    """bf16 activations with a few channels of each head larger than the rest, as projections have them."""
    x = torch.randn(n, heads, d, generator=g, device="cuda")
    if outliers:
        big = torch.rand(heads, d, generator=g, device="cuda") < 4.0 / d
        x = x * torch.where(big, 4.0, 1.0)
    return x.to(torch.bfloat16)


def _angles(n, rot, theta):
    """[n][rot] fp32: the cosines of the rot / 2 angles of each position, then their sines."""
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _quantise(x, group):
    """Codes, scales and zeros of x [...][d] in groups of `group` channels: fp32 x, fp16 scales and zeros."""
    y = x.unflatten(-1, (-1, group))
    lo, hi = y.amin(-1), y.amax(-1)
    s = ((hi - lo) / 15.0).half()
    z = lo.half()
    sf = s.float()[..., None]
    c = torch.where(sf > 0, torch.round((y - z.float()[..., None]) / sf), 0.0).clamp(0, 15)
    return c, s, z


def _pack(k, v, gk, gv):
    """The blocks of k, v [pages][16][heads][d] (fp32): [pages][heads][block bytes]."""
    p, _, h, d = k.shape
    w = d // 32
    kc, ks, kz = _quantise(k, gk)
    vc, vs, vz = _quantise(v, gv)
    kc = kc.flatten(-2).to(torch.uint8).permute(0, 2, 1, 3).reshape(p, h, PAGE, w, 4, 8).transpose(3, 4)
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(p, h, -1)
    vc = vc.flatten(-2).to(torch.uint8).permute(0, 2, 1, 3).reshape(p, h, 8, 2, w, 8, 4).permute(0, 1, 2, 5, 4, 3, 6)
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(p, h, -1)
    pairs = torch.cat([torch.stack([ks, kz], -1), torch.stack([vs, vz], -1)], 3)
    pairs = pairs.permute(0, 2, 1, 3, 4).reshape(p, h, -1).contiguous().view(torch.uint8)
    return torch.cat([kb, vb, pairs], -1)


def _table(case, g):
    """Page table [batch][pages of the longest] of a shuffled pool, -1 past each request's end; the pool's size."""
    pages = [-(-x // PAGE) for x in _contexts(case)]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _filled_pool(case, g, table, n_pages):
    """A pool whose pages hold quantised keys and values (every slot, so that slots past an end are stale, not zero)."""
    h, d = case["n_kv"], case["d"]
    pool = torch.empty(n_pages, h, PAGE * _packed(case), dtype=torch.uint8, device="cuda")
    at_once = max(1, (1 << 27) // (PAGE * h * d))
    for p in range(0, n_pages, at_once):
        n = min(at_once, n_pages - p)
        k = _rows(g, n * PAGE, h, d, True).float().reshape(n, PAGE, h, d)
        v = _rows(g, n * PAGE, h, d, False).float().reshape(n, PAGE, h, d)
        pool[p:p + n] = _pack(k, v, case["gk"], case["gv"])
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, b, h, d = "cuda", case["batch"], case["n_kv"], case["d"]
    lens, ctx = _lengths(case), _contexts(case)
    n = sum(lens)
    st = {"case": case, "lens": torch.tensor(ctx, dtype=torch.int32, device=dev)}
    if case["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["n_q"] + 1, device=dev) / case["n_q"]).float()
    if case["op"] == "prompt":
        def starts(x):
            return torch.tensor([sum(x[:i]) for i in range(b + 1)], dtype=torch.int32, device=dev)
        st.update(cu_q=starts(lens), cu_k=starts(ctx), max_q=max(lens), max_k=max(ctx),
                  q=_rows(g, n, case["n_q"], d, False), k=_rows(g, sum(ctx), h, d, True), v=_rows(g, sum(ctx), h, d, False),
                  prefix=torch.full((b,), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None)
        if own:
            _own_prompt(st)
        return st
    table, n_pages = _table(case, g)
    st.update(table=table, n_pages=n_pages, max_len=max(ctx))
    if case["op"] == "decode":
        st["q"] = _rows(g, b, case["n_q"], d, False)
        st["pool"] = _filled_pool(case, g, table, n_pages)
    else:
        st["req"] = torch.cat([torch.full((x,), i, dtype=torch.int32, device=dev) for i, x in enumerate(lens)])
        st["pos"] = torch.cat([torch.arange(c - x, c, dtype=torch.int32, device=dev) for x, c in zip(lens, ctx)])
        if case["op"] == "append":
            # one projection's output: the heads of q, k and v of a token side by side
            qkv = torch.cat([_rows(g, n, case["n_q"], d, False), _rows(g, n, h, d, True), _rows(g, n, h, d, False)], 1)
            st["q"], st["k"], st["v"] = qkv.split([case["n_q"], h, h], 1)
            st["angles"] = _angles(max(ctx), case["rot"], case["theta"])
        else:
            st["pool"] = _filled_pool(case, g, table, n_pages)
    if own:
        _own_cache(st)
    return st


# ------------------------------------------------------- the framework's calls

def _own_score(st):
    from bit_rotated_kv_split_gb300 import binding as B
    case = st["case"]
    return B.score_desc(softcap=case["cap"], window=case["window"], slopes=st.get("slopes"))


def _own_cache(st):
    """What a serving program keeps: the cache, its descriptor, the rotation's, and the decode's workspace."""
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    case = st["case"]
    cache = Int4Cache(case["batch"], case["n_q"], case["n_kv"], case["d"], st["table"].shape[1], st["n_pages"],
                      quant_group_k=case["gk"], quant_group_v=case["gv"])
    cache.page_table.copy_(st["table"])
    cache.seq_len.copy_(st["lens"])
    if "pool" in st:
        cache.pages.copy_(st.pop("pool").reshape(-1))
    st["cache"], st["desc"] = cache, cache.desc(st["max_len"])
    if case["op"] == "append":
        st["rope"] = B.rope_desc(st["angles"], case["rot"], case["interleaved"])
    if case["op"] == "decode":
        st["score"] = _own_score(st)
        st["ws"] = torch.zeros(B.oscar_decode_int4_workspace_bytes(st["desc"]), dtype=torch.uint8, device="cuda")


def _own_prompt(st):
    from bit_rotated_kv_split_gb300 import binding as B
    case = st["case"]
    st["desc"] = B.prompt_desc(case["batch"], case["n_q"], case["n_kv"], case["d"], st["max_q"], st["max_k"],
                               st["q"].shape[0], st["k"].shape[0], case["causal"])
    st["score"] = _own_score(st)
    st["ws"] = torch.zeros(B.oscar_prompt_workspace_bytes(st["desc"]), dtype=torch.uint8, device="cuda")


def _run_own(st):
    from bit_rotated_kv_split_gb300 import binding as B
    case = st["case"]
    op, d, h = case["op"], case["d"], case["n_kv"]
    if op == "prompt":
        out = torch.empty_like(st["q"])
        lse = torch.empty(out.shape[:2], dtype=torch.float32, device="cuda")
        B.oscar_prompt_attention(st["desc"], st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], out, st["ws"],
                                 score=st["score"], prefix_len=st["prefix"], lse=lse)
        return {"out": out, "lse": lse}
    if op == "decode":
        out = torch.empty_like(st["q"])
        B.oscar_decode_attention_int4(st["desc"], st["q"], out, st["ws"], score=st["score"])
        return {"out": out}
    n = st["req"].shape[0]
    got = {}
    if op == "append":
        got["q"] = torch.empty(n, case["n_q"], d, dtype=torch.bfloat16, device="cuda")
        got["k"] = torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda")
        B.oscar_rope_append_int4(st["desc"], st["rope"], st["q"], st["k"], st["v"], st["req"], st["pos"], got["q"], got["k"])
    got["cached_k"] = torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda")
    got["cached_v"] = torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda")
    B.oscar_gather_int4(st["desc"], st["req"], st["pos"], got["cached_k"], got["cached_v"])
    return got


# ------------------------------------------------------------- the plain forms

def _rotate(x, cs, interleaved):
    """x [n][heads][d] rotated by cs [n][rot]; in 64 bits, since the rounding to bf16 comes next and codes follow from it."""
    rot = cs.shape[1]
    c, s = cs.double()[:, None, :].chunk(2, -1)
    y = x.double()
    head, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        head = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([head, rest], -1).to(torch.bfloat16)


def _held(x, group):
    """What a row stands for once it is held in 4 bits."""
    c, s, z = _quantise(x.float().clamp(-65504.0, 65504.0), group)
    return (z.float()[..., None] + s.float()[..., None] * c).flatten(-2).to(torch.bfloat16)


def _unpack(blocks, case):
    """K and V [...][16][d] fp32 of blocks [...][block bytes]."""
    d, w = case["d"], case["d"] // 32
    ng = d // case["gk"]
    lead = blocks.shape[:-1]
    kb, vb, pairs = blocks.split([8 * d, 8 * d, blocks.shape[-1] - 16 * d], -1)
    k = torch.stack([kb & 15, kb >> 4], -1).reshape(*lead, PAGE, 4, w, 8).transpose(-3, -2).reshape(*lead, PAGE, d)
    v = torch.stack([vb & 15, vb >> 4], -1).reshape(*lead, 8, 8, w, 2, 4)
    v = v.movedim(-2, -4).transpose(-3, -2).reshape(*lead, PAGE, d)
    pairs = pairs.contiguous().view(torch.float16).reshape(*lead, PAGE, -1, 2).float()

    def value(c, p):
        c = c.float().unflatten(-1, (p.shape[-2], -1))
        return (p[..., 1:] + p[..., :1] * c).flatten(-2)
    return value(k, pairs[..., :ng, :]), value(v, pairs[..., ng:, :])


def _capped(t, case):
    return case["cap"] * torch.tanh(t / case["cap"]) if case["cap"] else t


def _attend(t, v):
    """Softmax of t [...][keys] (-inf where masked) against v [...][keys][d]; its logarithm of the sum. Rows with nothing give zeros."""
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return out, (m + torch.log(l)).squeeze(-1)


def _run_decode(st):
    case = st["case"]
    b, h, d = case["batch"], case["n_kv"], case["d"]
    k, v = _unpack(st["pool"][st["table"].clamp(min=0).long()], case)     # [b][pages][h][16][d]
    k = k.transpose(1, 2).reshape(b, h, -1, d)
    v = v.transpose(1, 2).reshape(b, h, -1, d)
    q = st["q"].float().reshape(b, h, -1, d)
    t = _capped(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d)), case)
    j = torch.arange(k.shape[2], device="cuda")
    gap = (j - (st["lens"].long()[:, None] - 1))[:, None, None]           # key minus query position
    if case["slopes"]:
        t = t + st["slopes"].reshape(1, h, -1, 1) * gap
    seen = gap <= 0
    if case["window"]:
        seen = seen & (gap > -case["window"])
    t = torch.where(seen, t, -math.inf)
    out, _ = _attend(t, torch.where((gap <= 0).squeeze(2)[..., None], v, 0.0))
    return {"out": out.reshape(b, -1, d).to(torch.bfloat16)}


def _run_prompt(st):
    case = st["case"]
    b, h, d, mq, mk = case["batch"], case["n_kv"], case["d"], st["max_q"], st["max_k"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    n_q, n_k = cu_q.diff(), cu_k.diff()
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    has_q, has_k = iq < n_q[:, None], ik < n_k[:, None]
    at_q = (cu_q[:-1, None] + iq).clamp(max=st["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=st["k"].shape[0] - 1)
    q = st["q"][at_q].float().reshape(b, mq, h, -1, d).permute(0, 2, 3, 1, 4)
    k = st["k"][at_k].float().permute(0, 2, 1, 3)[:, :, None]
    v = st["v"][at_k].float().permute(0, 2, 1, 3)[:, :, None]
    t = _capped(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d)), case)
    gap = ik - (iq + (n_k - n_q)[:, None])[..., None]                     # [b][mq][mk]
    if case["slopes"]:
        t = t - st["slopes"].reshape(1, h, -1, 1, 1) * gap.abs()[:, None, None]
    seen = torch.ones_like(gap, dtype=torch.bool)
    if case["causal"]:
        seen = gap <= 0
    if case["window"]:
        seen = seen & (gap > -case["window"])
    if case["prefix"]:
        seen = seen | (ik < st["prefix"].long()[:, None])[:, None]
    seen = seen & has_k[:, None]
    t = torch.where(seen[:, None, None], t, -math.inf)
    out, lse = _attend(t, v)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, mq, -1, d)[has_q]
    lse = lse.permute(0, 3, 1, 2).reshape(b, mq, -1)[has_q]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "decode":
        return _run_decode(state)
    if case["op"] == "prompt":
        return _run_prompt(state)
    if case["op"] == "append":
        cs = state["angles"][state["pos"].long()]
        k = _rotate(state["k"], cs, case["interleaved"])
        return {"q": _rotate(state["q"], cs, case["interleaved"]), "k": k, "cached_k": _held(k, case["gk"]),
                "cached_v": _held(state["v"], case["gv"])}
    req, pos = state["req"].long(), state["pos"].long()
    k, v = _unpack(state["pool"][state["table"].clamp(min=0).long()], case)   # [b][pages][h][16][d]
    return {"cached_k": k[req, pos // PAGE, :, pos % PAGE].to(torch.bfloat16),
            "cached_v": v[req, pos // PAGE, :, pos % PAGE].to(torch.bfloat16)}


# ----------------------------------------------- the definitions, in 64 bits

def _exact_values(pool, page, slot, case, which):
    """The float64 values [tokens][d] of KV head `which[0]`, K or V, of the tokens at (page, slot), nibble by nibble."""
    head, is_v = which
    d, w = case["d"], case["d"] // 32
    ch = torch.arange(d, device="cuda")
    t = slot[:, None]
    if is_v:
        word = (8 * (t // 2) + ch % 32 // 4) * w + ch // 32
        nibble = 4 * (t % 2) + ch % 4
        byte = 8 * d + 4 * word + nibble // 2
    else:
        word = w * (ch % 32 // 8) + ch // 32
        nibble = (ch % 8).expand(len(slot), d)
        byte = t * (d // 2) + 4 * word + nibble // 2
    block = pool[page, head]
    code = (block.gather(1, byte) >> (4 * (nibble % 2)).to(torch.uint8)) & 15
    ng, group = d // case["gk"], ch // (case["gv"] if is_v else case["gk"])
    at = 16 * d + 4 * ((ng + d // case["gv"]) * t + (ng if is_v else 0) + group)

    def half(o):
        bits = block.gather(1, at + o).int() | (block.gather(1, at + o + 1).int() << 8)
        return bits.to(torch.int16).view(torch.float16).double()
    return half(2) + half(0) * code.double()


def _exact_rows(x, cs, interleaved):
    n, heads, d = x.shape
    rot = cs.shape[1]
    y = x.double().clone()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(y[..., a], y[..., b]) * torch.complex(cs[:, :rot // 2].double(), cs[:, rot // 2:].double())[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_held(x, group):
    n, heads, d = x.shape
    y = x.double().clamp(-65504.0, 65504.0).reshape(n, heads, d // group, group)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    s, z = ((hi - lo) / 15).half().double(), lo.half().double()
    c = torch.nan_to_num((y - z) / s, nan=0.0, posinf=0.0, neginf=0.0).round().clamp(0, 15)
    return (z + s * c).reshape(n, heads, d)


def _exact_attend(q, k, v, case, slopes, n_k, first_q, prefix):
    """Attention of q [n][d] (positions first_q ..) over k, v [n_k][d], all float64: (out, logarithm of the sum)."""
    t = q @ k.T / math.sqrt(case["d"])
    if case["cap"]:
        t = torch.tanh(t / case["cap"]) * case["cap"]
    i = torch.arange(first_q, first_q + q.shape[0], device="cuda")[:, None]
    j = torch.arange(n_k, device="cuda")[None]
    if slopes is not None:
        t = t - slopes * (i - j).abs()
    hidden = (j > i) if case["causal"] else torch.zeros_like(t, dtype=torch.bool)
    if case["window"]:
        hidden = hidden | (i - j >= case["window"])
    if prefix:
        hidden = hidden & (j >= prefix)
    t = t.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(t, 1)
    p = torch.exp(t - torch.where(lse.isfinite(), lse, 0.0)[:, None])
    return p @ v, lse


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op, h, d = case["op"], case["n_kv"], case["d"]
    group = case["n_q"] // h
    slopes = st["slopes"].double() if case["slopes"] else [None] * case["n_q"]
    if op == "append":
        cs = st["angles"][st["pos"].long()]
        k = _exact_rows(st["k"], cs, case["interleaved"])
        # the cache holds the rounded row
        return {"q": _exact_rows(st["q"], cs, case["interleaved"]), "k": k, "cached_k": _exact_held(k.to(torch.bfloat16), case["gk"]),
                "cached_v": _exact_held(st["v"], case["gv"])}
    if op == "read":
        page = st["table"][st["req"].long(), st["pos"].long() // PAGE].long()
        slot = st["pos"].long() % PAGE
        return {name: torch.stack([_exact_values(st["pool"], page, slot, case, (x, is_v)) for x in range(h)], 1)
                for name, is_v in (("cached_k", False), ("cached_v", True))}
    if op == "decode":
        out = torch.zeros(case["batch"], case["n_q"], d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens"].tolist()):
            at = torch.arange(n, device="cuda")
            page, slot = st["table"][b].long()[at // PAGE], at % PAGE
            for x in range(h):
                k, v = (_exact_values(st["pool"], page, slot, case, (x, is_v)) for is_v in (False, True))
                for q in range(x * group, (x + 1) * group):
                    out[b, q] = _exact_attend(st["q"][b, q:q + 1].double(), k, v, case, slopes[q], n, n - 1, 0)[0][0]
        return {"out": out}
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(case["batch"]):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, n_k = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for q in range(case["n_q"]):
            k, v = st["k"][keys, q // group].double(), st["v"][keys, q // group].double()
            out[rows, q], lse[rows, q] = _exact_attend(st["q"][rows, q].double(), k, v, case, slopes[q], n_k, n_k - n, min(case["prefix"], n_k))
    return {"out": out, "lse": lse}
