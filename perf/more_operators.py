"""The operators of a layer whose KV cache is held in 8 bits, and of rotary positions, as measured workloads.

Five operators: filling a table of rotation angles whose frequencies are scaled
for long contexts ("table"), norm and rotation of a projection's query and key
heads ("rope"), the same with the keys and values quantised and written to the
paged 8-bit cache ("append"), reading cached rows back as bf16 ("read") and
attention of one query token per request over the cache ("decode").  Each in its
plain form (elementary torch operations) and, where `own` is true, as calls of
this repository's library.

A vector of d channels is held as d codes 0 .. 255 and an fp16 (scale, zero):
zero is its least value rounded down, scale (greatest - zero) / 255 rounded up,
and a channel stands for zero + scale * code.  A block of one (page, KV head)
holds 16 tokens of head size d, 64 or 128:
  [0, 16 d)     K codes: channel 16 c + i of token t is byte
                t d + 16 (c ^ x) + i, x = t % 8 (d = 128) or t / 2 % 4 (d = 64);
  [16 d, 32 d)  V codes, the same way;
  [32 d, ...)   token t's K scale, K zero, V scale, V zero (fp16) at 32 d + 8 t.
"""
import math

import torch

own = False

PAGE = 16
TAU = 65504.0


# ------------------------------------------------------------------- the cases

def _case(name, op, batch=1, lo=1, hi=1, n_q=32, n_kv=8, d=128, past=0, rot=128, interleaved=False, norm=False, theta=1e6,
          kind="none", factor=1.0, original=32_768, cap=0.0, window=0, slopes=False):
    c = dict(name=name, op=op, batch=batch, lo=lo, hi=hi, n_q=n_q, n_kv=n_kv, d=d, past=past, rot=rot, interleaved=interleaved,
             norm=norm, theta=theta, kind=kind, factor=factor, original=original, cap=cap, window=window, slopes=slopes)
    if not name:
        del c["name"]
    return c


def listed():
    return [
        # angles of a short context, plain frequencies, half of each head: what a server with small models makes at its start
        _case("table-4k", "table", hi=4_099, rot=64, theta=1e4),
        # angles of a million positions, frequencies scaled by parts for a context longer than the trained one
        _case("table-1m", "table", hi=1_048_576, rot=128, theta=1e6, kind="index", factor=4.0),
        # the new tokens of a serving batch of odd size: norm and rotation of q and k for a layer that quantises elsewhere
        _case("rope-61-tokens", "rope", 61, 1, 1, 64, 8, 128, past=20_000, rot=64, interleaved=True, norm=True, theta=1e4),
        # whole prompts of different lengths, 30k tokens together
        _case("rope-prompts", "rope", 5, 2_113, 12_001, 32, 8, 128, rot=128, norm=True, kind="linear", factor=2.0),
        # one new token of one request, deep in its context: what a decode step adds; latency is all
        _case("append-1-token", "append", 1, 1, 1, 32, 8, 128, past=99_999, rot=128, norm=True),
        # whole prompts, 30k tokens together: prefill
        _case("append-prompts", "append", 5, 2_113, 12_001, 32, 8, 128, rot=128, norm=True, kind="wave", factor=8.0),
        # a short shared prefix read back, small heads
        _case("read-short", "read", 3, 97, 501, 16, 4, 64),
        # a long cached prefix read back, so that a prompt can go on from it
        _case("read-prefix", "read", 1, 65_521, 65_521, 32, 8, 128),
        # single tokens: a chat's short context, one request
        _case("decode-1x777", "decode", 1, 777, 777, 32, 8, 128),
        # one request of 100k tokens
        _case("decode-1x100k", "decode", 1, 100_000, 100_000, 32, 8, 128),
        # a ragged batch, GQA 8, capped scores
        _case("decode-28-ragged-cap", "decode", 28, 2_000, 32_000, 64, 8, 128, cap=50.0),
        # small heads, a group of five, a bias by distance within a window
        _case("decode-16-bias-window", "decode", 16, 301, 9_001, 40, 8, 64, window=4_096, slopes=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "read", "decode"])
    d = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    while n_q > 64:
        n_q -= n_kv
    kind = rng.choice(["none", "linear", "base", "index", "wave"])
    angles = dict(rot=rng.choice([16, d // 2, d]), theta=rng.choice([1e4, 1e6]), kind=kind,
                  factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([4_096, 8_192, 32_768]))
    if op == "table":
        return _case("", op, hi=_log_int(rng, 16, 1_000_000), d=d, **angles)
    if op in ("rope", "append"):
        n = _log_int(rng, 1, 29_000 * 32 // max(n_q, 32))
        batch = min(n, _log_int(rng, 1, 200))
        hi = max(1, n // batch)
        return _case("", op, batch, max(1, hi - rng.randrange(0, hi)), hi, n_q, n_kv, d, past=rng.choice([0, _log_int(rng, 1, 100_000)]),
                     interleaved=rng.random() < 0.5, norm=rng.random() < 0.6, **angles)
    if op == "read":
        n = _log_int(rng, 1, 60_000)
        batch = min(n, _log_int(rng, 1, 200))
        hi = max(1, n // batch)
        return _case("", op, batch, max(1, hi - rng.randrange(0, hi)), hi, n_q, n_kv, d)
    total = _log_int(rng, 100, 300_000)     # tokens of all requests
    batch = min(total, _log_int(rng, 1, 128))
    hi = max(1, total // batch)
    return _case("", op, batch, max(1, hi // rng.choice([1, 2, 7])), hi, n_q, n_kv, d, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                 window=rng.choice([0, 0, _log_int(rng, 16, 8_000)]), slopes=rng.random() < 0.3)


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


def work(case):
    n, d, n_q, n_kv, rot = sum(_lengths(case)), case["d"], case["n_q"], case["n_kv"], case["rot"]
    held = 2 * (d + 4)                      # bytes of one token of one KV head in the cache, K and V together
    if case["op"] == "table":               # the two powers of a pair: about seven products each
        return {"bytes": 4 * case["hi"] * rot, "flops": 15.0 * case["hi"] * rot}
    norm = 4.0 * d if case["norm"] else 0.0
    if case["op"] == "rope":
        return {"bytes": 4 * d * n * (n_q + n_kv) + 4 * n * rot, "flops": n * (n_q + n_kv) * (3.0 * rot + norm)}
    if case["op"] == "append":              # the rows in, the rotated queries out, the codes out, and what they stand for
        return {"bytes": 2 * d * n * (2 * n_q + 4 * n_kv) + n * n_kv * held + 4 * n * rot,
                "flops": n * (n_q + n_kv) * (3.0 * rot + norm) + 12.0 * n * n_kv * d}
    if case["op"] == "read":
        return {"bytes": n * n_kv * (held + 4 * d), "flops": 4.0 * n * n_kv * d}
    seen = sum(min(x, case["window"] or x) for x in _lengths(case))
    return {"bytes": seen * n_kv * held + 4 * d * n_q * case["batch"] + 4 * n_q * case["batch"], "flops": 4.0 * seen * n_q * d}


# ------------------------------------------------------------------ the inputs

def _rows(g, n, heads, d, outliers):
    """bf16 activations with a few channels of each head larger than the rest, as projections have them."""
    x = torch.randn(n, heads, d, generator=g, device="cuda")
    if outliers:
        big = torch.rand(heads, d, generator=g, device="cuda") < 4.0 / d
        x = x * torch.where(big, 4.0, 1.0)
    return x.to(torch.bfloat16)


def _frequencies(case):
    """(radians per position of each pair [rot / 2] float64, the factor on cosines and sines)."""
    rot, theta, f, original = case["rot"], case["theta"], case["factor"], case["original"]
    if case["kind"] == "base":              # a larger base: the fastest pair keeps its frequency, the slowest gets 1 / f
        theta = theta * f ** (rot / max(rot - 2, 1))
    w = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["kind"] == "linear":
        return w / f, 1.0
    turns = original * w / (2.0 * math.pi)  # of each pair over the trained context
    if case["kind"] == "index":             # pairs of over 32 turns stay, of under 1 are slowed, a ramp over their index between
        def at(r):
            return rot * math.log(original / (r * 2.0 * math.pi)) / (2.0 * math.log(theta))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        keep = 1.0 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w * keep + w / f * (1.0 - keep), 0.1 * math.log(f) + 1.0
    if case["kind"] == "wave":              # pairs of over 4 turns stay, of under 1 are slowed, a ramp over their turns between
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return w * keep + w / f * (1.0 - keep), 1.0
    return w, 1.0


def _turned(w, magnitude, n):
    """[n][rot] fp32: the cosines of the angles of each position, then their sines; the angles in 64 bits."""
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * w.to("cuda")
    return torch.cat([a.cos() * magnitude, a.sin() * magnitude], 1).float()


def _step(h, up):
    """The fp16 number next to h, above or below."""
    bits = h.view(torch.int16).int()
    key = torch.where(bits < 0, -(bits & 0x7FFF), bits) + (1 if up else -1)
    return torch.where(key < 0, -32768 - key, key).to(torch.int16).view(torch.float16)


def _quantise(x):
    """Codes, scales and zeros of x [...][d]: float64 codes, fp16 scales and zeros."""
    y = x.double()
    lo, hi = y.amin(-1), y.amax(-1)
    z = lo.half()
    z = torch.where(z.double() > lo, _step(z, False), z)
    t = (hi - z.double()) / 255.0
    s = t.half()
    s = torch.where(s.double() < t, _step(s, True), s)
    sd = s.double()[..., None]
    return torch.where(sd > 0, torch.round((y - z.double()[..., None]) / torch.where(sd > 0, sd, 1.0)), 0.0), s, z


def _swizzled(c):
    """Rows [...][16][d] of bytes with their 16-byte chunks at the places that a block has them (its own inverse)."""
    d = c.shape[-1]
    t = torch.arange(PAGE, device=c.device)[:, None]
    chunk = torch.arange(d // 16, device=c.device) ^ (t % 8 if d == 128 else t // 2 % 4)
    at = (16 * chunk[..., None] + torch.arange(16, device=c.device)).flatten(-2)
    return c.gather(-1, at.expand(c.shape))


def _pack(k, v):
    """The blocks of k, v [pages][16][heads][d]: [pages][heads][block bytes]."""
    kc, ks, kz = _quantise(k.transpose(1, 2))
    vc, vs, vz = _quantise(v.transpose(1, 2))
    pairs = torch.stack([ks, kz, vs, vz], -1).contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([_swizzled(kc.to(torch.uint8)).flatten(-2), _swizzled(vc.to(torch.uint8)).flatten(-2), pairs], -1)


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


def _filled_pool(case, g, n_pages):
    """A pool whose pages hold quantised keys and values (every slot, so that slots past an end are stale, not zero)."""
    h, d = case["n_kv"], case["d"]
    pool = torch.empty(n_pages, h, PAGE * (2 * d + 8), dtype=torch.uint8, device="cuda")
    at_once = max(1, (1 << 27) // (PAGE * h * d))
    for p in range(0, n_pages, at_once):
        n = min(at_once, n_pages - p)
        k = _rows(g, n * PAGE, h, d, True).reshape(n, PAGE, h, d)
        v = _rows(g, n * PAGE, h, d, False).reshape(n, PAGE, h, d)
        pool[p:p + n] = _pack(k, v)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, b, h, d, op = "cuda", case["batch"], case["n_kv"], case["d"], case["op"]
    lens, ctx = _lengths(case), _contexts(case)
    n = sum(lens)
    st = {"case": case}
    w, magnitude = _frequencies(case)
    if op == "table":                       # another seed: a slightly different base
        st["w"] = w * (1.0 - 1e-3 * float(torch.rand(1, generator=g, device=dev)))
        st["magnitude"] = magnitude
        st["out"] = torch.empty(case["hi"], case["rot"], dtype=torch.float32, device=dev)
        return st
    st["req"] = torch.cat([torch.full((x,), i, dtype=torch.int32, device=dev) for i, x in enumerate(lens)])
    st["pos"] = torch.cat([torch.arange(c - x, c, dtype=torch.int32, device=dev) for x, c in zip(lens, ctx)])
    if op in ("rope", "append"):
        # one projection's output: the heads of q, k and v of a token side by side
        qkv = torch.cat([_rows(g, n, case["n_q"], d, False), _rows(g, n, h, d, True), _rows(g, n, h, d, False)], 1)
        st["q"], st["k"], st["v"] = qkv.split([case["n_q"], h, h], 1)
        st["angles"] = _turned(w, magnitude, max(ctx))
        if case["norm"]:
            st["wq"], st["wk"] = (1.0 + 0.2 * torch.randn(2, d, generator=g, device=dev)).to(torch.bfloat16)
    if op != "decode":
        st["q_out"] = torch.empty(n, case["n_q"], d, dtype=torch.bfloat16, device=dev)
        st["k_out"], st["v_out"] = (torch.empty(n, h, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if op == "rope":
        if own:
            _own_angles(st)
        return st
    st["lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    st["table"], n_pages = _table(case, g)
    st["n_pages"], st["max_len"] = n_pages, max(ctx)
    if op != "append":
        st["pool"] = _filled_pool(case, g, n_pages)
    if op == "decode":
        st["q"] = _rows(g, b, case["n_q"], d, False)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(b, case["n_q"], dtype=torch.float32, device=dev)
        if case["slopes"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["n_q"] + 1, device=dev) / case["n_q"]).float()
    if own:
        _own_cache(st)
    return st


# ------------------------------------------------------- the framework's calls

def _own_angles(st):
    from bit_rotated_kv_split_gb300 import binding as B
    case = st["case"]
    st["rope"] = B.rope_desc(st["angles"], case["rot"], case["interleaved"])
    st["norm"] = B.norm_desc(st["wq"], st["wk"], 1e-6) if case["norm"] else None


def _own_cache(st):
    """What a serving program keeps: the cache, its descriptor, the rotation's, and the decode's workspace."""
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int8Cache
    case = st["case"]
    cache = Int8Cache(case["batch"], case["n_q"], case["n_kv"], case["d"], st["table"].shape[1], st["n_pages"])
    cache.page_table.copy_(st["table"])
    cache.seq_len.copy_(st["lens"])
    if "pool" in st:
        cache.pages.copy_(st.pop("pool").reshape(-1))
    st["cache"], st["desc"] = cache, cache.desc(st["max_len"])
    if case["op"] == "append":
        _own_angles(st)
    if case["op"] == "decode":
        st["score"] = B.score_desc(softcap=case["cap"], window=case["window"], slopes=st.get("slopes"))
        st["ws"] = torch.zeros(B.oscar_decode_int8_workspace_bytes(st["desc"]), dtype=torch.uint8, device="cuda")


def _run_own(st):
    from bit_rotated_kv_split_gb300 import binding as B
    op = st["case"]["op"]
    if op == "table":
        B.oscar_rope_table(st["w"].numpy(), st["out"], magnitude=st["magnitude"])
        return {"cos_sin": st["out"]}
    if op == "rope":
        B.oscar_norm_rope(st["norm"], st["rope"], st["q"], st["k"], st["pos"], st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "append":
        B.oscar_rope_append_int8(st["desc"], st["norm"], st["rope"], st["q"], st["k"], st["v"], st["req"], st["pos"], st["q_out"],
                                 k_held=st["k_out"], v_held=st["v_out"])
        return {"q": st["q_out"], "cached_k": st["k_out"], "cached_v": st["v_out"]}
    if op == "read":
        B.oscar_gather_int8(st["desc"], st["req"], st["pos"], st["k_out"], st["v_out"])
        return {"cached_k": st["k_out"], "cached_v": st["v_out"]}
    B.oscar_decode_attention_int8(st["desc"], st["q"], st["out"], st["ws"], score=st["score"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------- the plain forms

def _norm_rotate(x, weight, cs, interleaved):
    """x [n][heads][d]: each head normed (where there is a weight), then rotated by cs [n][rot]; rounded once."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = cs.shape[1]
    c, s = cs[:, None, :].chunk(2, -1)
    head, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        head = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([head, rest], -1).to(torch.bfloat16)


def _held(x):
    """What rows stand for once they are held in 8 bits."""
    c, s, z = _quantise(x.float().clamp(-TAU, TAU))
    return (z.float()[..., None] + s.float()[..., None] * c.float()).to(torch.bfloat16)


def _unpack(blocks, d):
    """K and V [...][16][d] fp32 of blocks [...][block bytes]."""
    lead = blocks.shape[:-1]
    kc, vc, pairs = blocks.split([PAGE * d, PAGE * d, 8 * PAGE], -1)
    pairs = pairs.contiguous().view(torch.float16).reshape(*lead, PAGE, 4, 1).float()
    k = pairs[..., 1, :] + pairs[..., 0, :] * _swizzled(kc.reshape(*lead, PAGE, d)).float()
    v = pairs[..., 3, :] + pairs[..., 2, :] * _swizzled(vc.reshape(*lead, PAGE, d)).float()
    return k, v


def _run_decode(st):
    case = st["case"]
    b, h, d = case["batch"], case["n_kv"], case["d"]
    k, v = _unpack(st["pool"][st["table"].clamp(min=0).long()], d)        # [b][pages][h][16][d]
    k = k.transpose(1, 2).reshape(b, h, -1, d)
    v = v.transpose(1, 2).reshape(b, h, -1, d)
    q = st["q"].float().reshape(b, h, -1, d)
    t = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    if case["cap"]:
        t = case["cap"] * torch.tanh(t / case["cap"])
    gap = (torch.arange(k.shape[2], device="cuda") - (st["lens"].long()[:, None] - 1))[:, None, None]   # key minus query position
    if case["slopes"]:
        t = t + st["slopes"].reshape(1, h, -1, 1) * gap
    seen = gap <= 0
    if case["window"]:
        seen = seen & (gap > -case["window"])
    t = torch.where(seen, t, -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, torch.where((gap <= 0).squeeze(2)[..., None], v, 0.0)) / l
    return {"out": out.reshape(b, -1, d).to(torch.bfloat16), "lse": (m + torch.log(l)).reshape(b, -1)}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "table":
        return {"cos_sin": _turned(state["w"], state["magnitude"], case["hi"])}
    if op == "decode":
        return _run_decode(state)
    if op == "read":
        req, pos = state["req"].long(), state["pos"].long()
        k, v = _unpack(state["pool"][state["table"].clamp(min=0).long()], case["d"])   # [b][pages][h][16][d]
        return {"cached_k": k[req, pos // PAGE, :, pos % PAGE].to(torch.bfloat16),
                "cached_v": v[req, pos // PAGE, :, pos % PAGE].to(torch.bfloat16)}
    cs = state["angles"][state["pos"].long()]
    q = _norm_rotate(state["q"], state.get("wq"), cs, case["interleaved"])
    k = _norm_rotate(state["k"], state.get("wk"), cs, case["interleaved"])
    if op == "rope":
        return {"q": q, "k": k}
    return {"q": q, "cached_k": _held(k), "cached_v": _held(state["v"])}


# ----------------------------------------------- the definitions, in 64 bits

def _exact_rows(x, weight, cs, interleaved):
    n, heads, d = x.shape
    rot = cs.shape[1]
    y = x.double().clone()
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * weight.double()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(y[..., a], y[..., b]) * torch.complex(cs[:, :rot // 2].double(), cs[:, rot // 2:].double())[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _half_towards(x, up):
    """x rounded up or down to a multiple of fp16's step at its size, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))).clamp(min=-14.0) - 10.0)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def _exact_held(x):
    y = x.double().clamp(-TAU, TAU)
    z = _half_towards(y.min(-1, keepdim=True).values, False)
    s = _half_towards((y.max(-1, keepdim=True).values - z) / 255.0, True)
    return z + s * torch.nan_to_num((y - z) / s, nan=0.0, posinf=0.0, neginf=0.0).round()


def _exact_values(pool, page, slot, case, head, is_v):
    """The float64 values [tokens][d] of one KV head, K or V, of the tokens at (page, slot), byte by byte."""
    d = case["d"]
    ch = torch.arange(d, device="cuda")
    t = slot[:, None]
    x = t % 8 if d == 128 else t // 2 % 4
    block = pool[page, head]
    code = block.gather(1, (PAGE * d if is_v else 0) + t * d + 16 * (ch // 16 ^ x) + ch % 16)

    def half(o):
        at = 32 * d + 8 * t + (4 if is_v else 0) + o
        bits = block.gather(1, at).int() | (block.gather(1, at + 1).int() << 8)
        return bits.to(torch.int16).view(torch.float16).double()
    return half(2) + half(0) * code.double()


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op, h, d = case["op"], case["n_kv"], case["d"]
    if op == "table":
        turns = (torch.arange(case["hi"], dtype=torch.float64, device="cuda")[:, None] * (st["w"] / (2.0 * math.pi)).to("cuda")).frac()
        z = torch.polar(torch.full_like(turns, st["magnitude"]), turns * (2.0 * math.pi))
        return {"cos_sin": torch.cat([z.real, z.imag], 1)}
    if op in ("rope", "append"):
        cs = st["angles"][st["pos"].long()]
        q, k = (_exact_rows(st[x], st.get("w" + x), cs, case["interleaved"]) for x in "qk")
        if op == "rope":
            return {"q": q, "k": k}
        return {"q": q, "cached_k": _exact_held(k.to(torch.bfloat16)), "cached_v": _exact_held(st["v"])}   # the cache holds the rounded row
    if op == "read":
        page = st["table"][st["req"].long(), st["pos"].long() // PAGE].long()
        slot = st["pos"].long() % PAGE
        return {name: torch.stack([_exact_values(st["pool"], page, slot, case, x, is_v) for x in range(h)], 1)
                for name, is_v in (("cached_k", False), ("cached_v", True))}
    group = case["n_q"] // h
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        at = torch.arange(n, device="cuda")
        page, slot = st["table"][b].long()[at // PAGE], at % PAGE
        for x in range(h):
            heads = slice(x * group, (x + 1) * group)
            k, v = (_exact_values(st["pool"], page, slot, case, x, is_v) for is_v in (False, True))
            t = st["q"][b, heads].double() @ k.T / math.sqrt(d)
            if case["cap"]:
                t = torch.tanh(t / case["cap"]) * case["cap"]
            if case["slopes"]:
                t = t - st["slopes"][heads, None].double() * (n - 1 - at)
            if case["window"]:
                t = t.masked_fill(at <= n - 1 - case["window"], -math.inf)
            lse[b, heads] = torch.logsumexp(t, 1)
            out[b, heads] = torch.softmax(t, 1) @ v
    return {"out": out, "lse": lse}
