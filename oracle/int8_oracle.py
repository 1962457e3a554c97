"""Float64 oracle of the 8-bit layers and of rotary positions (plain numpy).

Shares no code with the CUDA library and none with the measured workloads.
An 8-bit layer's vector of d channels is 256 codes and one fp16 (scale, zero):
zero is the least channel rounded down, scale (greatest - zero) / 255 rounded
up.  Pages of 16 tokens, one block of 32 d + 128 bytes per (page, KV head):
  K codes: channel 16 c + i of slot t at t d + 16 (c ^ x) + i, x = t % 8
    (d = 128) or (t // 2) % 4 (d = 64); V codes the same way from 16 d;
  slot t's K scale, K zero, V scale, V zero (fp16) at 32 d + 8 t.
"""
from __future__ import annotations

import math

import numpy as np

PAGE8 = 16


def int8_block_bytes(d: int) -> int:
    return 32 * d + 128


def half_towards(x, up: bool) -> np.ndarray:
    """x (float64, in fp16's range) rounded up or down to fp16."""
    x = np.asarray(x, dtype=np.float64)
    h = x.astype(np.float16)
    off = h.astype(np.float64) < x if up else h.astype(np.float64) > x
    with np.errstate(over="ignore"):
        return np.where(off, np.nextafter(h, np.float16(np.inf if up else -np.inf)), h)


def int8_quantize(x, tau: float = 65504.0):
    """(codes [...][d] uint8, scale [...] fp16, zero [...] fp16) of x clamped to [-tau, tau]."""
    x = np.clip(np.asarray(x, dtype=np.float64), -tau, tau)
    z = half_towards(x.min(-1), False)
    s = half_towards((x.max(-1) - z.astype(np.float64)) / 255.0, True)
    s64, z64 = s.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    u = np.divide(x - z64, s64, out=np.zeros_like(x), where=s64 > 0)
    return np.rint(u).astype(np.uint8), s, z


def int8_values(codes, s, z) -> np.ndarray:
    """zero + scale * code, float64."""
    return z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * codes.astype(np.float64)


def int8_code_byte(d: int, which: int, slot, ch):
    """Byte of channel ch of a slot's K (0) or V (1) in a block."""
    x = slot % 8 if d == 128 else slot // 2 % 4
    return 16 * d * which + slot * d + 16 * ((ch // 16) ^ x) + ch % 16


def int8_store_rows(pool: np.ndarray, pages, slots, which: int, codes, s, z) -> None:
    """Tokens at (pages[i], slots[i]), distinct, into pool [pages][n_kv][block]: codes [T][n_kv][d], s and z [T][n_kv]."""
    t, h, d = codes.shape
    pages, slots = np.asarray(pages)[:, None], np.asarray(slots)[:, None]
    head = np.arange(h)[None]
    pool[pages[..., None], head[..., None], int8_code_byte(d, which, slots, np.arange(d)[None])[:, None]] = codes
    raw = np.stack([s, z], -1).astype(np.float16).view(np.uint8)
    for i in range(4):
        pool[pages, head, 32 * d + 8 * slots + 4 * which + i] = raw[..., i]


def int8_load(pool: np.ndarray, pages, slots, which: int, d: int):
    """(codes [T][n_kv][d], s, z [T][n_kv]) of the tokens at (pages[i], slots[i])."""
    blocks = pool[np.asarray(pages)]
    t, h = blocks.shape[:2]
    slots = np.asarray(slots)[:, None]
    at = int8_code_byte(d, which, slots, np.arange(d)[None])
    codes = np.take_along_axis(blocks, np.broadcast_to(at[:, None], (t, h, d)), 2)
    o = 32 * d + 8 * slots + 4 * which
    raw = np.stack([np.take_along_axis(blocks, np.broadcast_to((o + i)[:, None], (t, h, 1)), 2)[..., 0] for i in range(4)], -1)
    sz = np.ascontiguousarray(raw).view(np.float16)
    return codes, sz[..., 0], sz[..., 1]


def head_norm(x, weight, eps: float) -> np.ndarray:
    """x [...][d] / sqrt(mean of squares + eps) * weight, float64 (weight None: x)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps) * np.asarray(weight, dtype=np.float64)


def rope_frequencies(rot: int, theta: float, kind: str = "plain", factor: float = 1.0, original: float = 0.0,
                     low: float = 1.0, high: float = 1.0):
    """(radians per position of each pair, magnitude), by the definitions of the kinds."""
    out = []
    if kind == "base":
        theta = theta * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        slow = w / factor
        turns = original * w / (2 * math.pi)
        if kind == "linear":
            w = slow
        elif kind == "by_turns":
            part = min(max((high - turns) / (high - low), 0.0), 1.0)
            w = slow * part + w * (1 - part)
        elif kind == "by_index":
            def index(r):       # of the pair that makes r turns: theta^(-2 i / rot) original / 2 pi = r
                return math.log(original / (2 * math.pi * r), theta) * rot / 2
            a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
            part = min(max((i - a) / (b - a if b > a else 1e-3), 0.0), 1.0)
            w = slow * part + w * (1 - part)
        out.append(w)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if kind == "by_index" else 1.0)


def rope_table(freq, first: int, n: int, magnitude: float = 1.0) -> np.ndarray:
    """[n][2 len(freq)] float64 cosines and sines; the products and the reduction by whole turns in extended precision."""
    turns = []
    scale = 1 << 200
    # 2 pi to 60 digits, as an integer over 10^60
    two_pi = 6283185307179586476925286766559005768394338798750211641949889
    for w in np.asarray(freq, dtype=np.float64):
        num, den = float(w).as_integer_ratio()
        one = num * 10 ** 60 * scale // (den * two_pi)      # turns of one position, over 2^200
        turns.append([((first + j) * one % scale) / scale for j in range(n)])
    a = np.array(turns).T.reshape(n, len(turns))
    # the first octant's angle with its sign and quarter, so that small sines keep their bits
    q = np.rint(a * 4)
    r = (a * 4 - q) * (math.pi / 2)
    q = q.astype(int) % 4
    s, c = np.sin(r), np.cos(r)
    sine = np.choose(q, [s, c, -s, -c])
    cosine = np.choose(q, [c, -s, -c, s])
    return np.concatenate([cosine, sine], 1) * magnitude
