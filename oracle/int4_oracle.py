"""Float64 oracle of the 4-bit layers and of prompt attention (plain numpy).

Shares no code with the CUDA library and none with the measured workloads.
The 4-bit layer is this library's format: fp16 (scale, zero) per group of
channels and sixteen codes; pages of 16 tokens, one block per (page, KV head)
of d channels, W = d / 32:
  K codes at [0, 8 d): slot t's bytes at t d / 2, channel 32 w + 8 u + n is
    nibble n of 32-bit word W u + w;
  V codes at [8 d, 16 d): channel 32 w + 4 u + n of slot t is nibble
    4 (t % 2) + n of word (8 (t // 2) + u) W + w;
  pairs at 16 d: slot t's K pairs, then its V pairs, (scale, zero) fp16.
"""
from __future__ import annotations

import numpy as np

PAGE = 16


def bf16(x) -> np.ndarray:
    """x rounded to float32, then to bfloat16 (nearest even), as float64.  Finite x."""
    b = np.asarray(x, dtype=np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def int4_block_bytes(d: int, ng_k: int, ng_v: int) -> int:
    return 16 * d + 64 * (ng_k + ng_v)


def int4_quantize(x, group: int, tau: float):
    """(codes [...][d] uint8, scale [...][d/g] fp16, zero [...][d/g] fp16) of x clamped to [-tau, tau]."""
    x = np.clip(np.asarray(x, dtype=np.float64), -tau, tau)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    lo, hi = y.min(-1), y.max(-1)
    s = ((hi - lo) / 15.0).astype(np.float16)
    z = lo.astype(np.float16)
    s64, z64 = s.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    u = np.divide(y - z64, s64, out=np.zeros_like(y), where=s64 > 0)
    c = np.clip(np.rint(u), 0, 15).astype(np.uint8)
    return c.reshape(x.shape), s, z


def int4_values(codes, s, z) -> np.ndarray:
    """zero + scale * code, float64."""
    c = codes.reshape(s.shape + (codes.shape[-1] // s.shape[-1],)).astype(np.float64)
    v = z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * c
    return v.reshape(codes.shape)


def _nibble(d: int, which: int, slot, ch):
    """(byte offset in a block, shift) of channel ch of a slot."""
    w = d // 32
    if which == 0:
        word, n = w * (ch % 32 // 8) + ch // 32, ch % 8
        return slot * (d // 2) + 4 * word + n // 2, 4 * (n % 2)
    word, n = (8 * (slot // 2) + ch % 32 // 4) * w + ch // 32, 4 * (slot % 2) + ch % 4
    return 8 * d + 4 * word + n // 2, 4 * (n % 2)


def _pair(d: int, ng_k: int, ng_v: int, which: int, slot, g):
    return 16 * d + 4 * ((ng_k + ng_v) * slot + (ng_k if which else 0) + g)


def int4_store(pool: np.ndarray, page: int, slot: int, which: int, codes, s, z, ng_k: int, ng_v: int) -> None:
    """One token of all KV heads into pool [pages][n_kv][block]: codes [n_kv][d], s and z [n_kv][groups]."""
    d = codes.shape[-1]
    ch = np.arange(d)
    at, sh = _nibble(d, which, slot, ch)
    for h in range(codes.shape[0]):
        block = pool[page, h]
        for a, b, c in zip(at, sh, codes[h]):
            block[a] = (int(block[a]) & (0xF0 if b == 0 else 0x0F)) | (int(c) << int(b))
        for g in range(s.shape[1]):
            o = _pair(d, ng_k, ng_v, which, slot, g)
            block[o:o + 4] = np.array([s[h, g], z[h, g]], np.float16).view(np.uint8)


def int4_store_rows(pool: np.ndarray, pages, slots, which: int, codes, s, z, ng_k: int, ng_v: int) -> None:
    """Tokens at (pages[i], slots[i]), distinct: codes [T][n_kv][d], s and z [T][n_kv][groups]."""
    t, h, d = codes.shape
    if t == 0:
        return
    pages, slots = np.asarray(pages)[:, None, None], np.asarray(slots)
    head = np.arange(h)[None, :, None]
    at, sh = _nibble(d, which, slots[:, None], np.arange(d)[None])
    sh = np.broadcast_to(sh, (t, d))
    for low in (True, False):               # a byte's two nibbles one after the other
        pick = sh[0] == (0 if low else 4)
        a, c = at[:, None, pick], codes[:, :, pick]
        old = pool[pages, head, a]
        pool[pages, head, a] = (old & 0xF0) | c if low else (old & 0x0F) | (c << 4)
    for g in range(s.shape[2]):
        o = _pair(d, ng_k, ng_v, which, slots, g)[:, None]
        raw = np.stack([s[:, :, g], z[:, :, g]], -1).astype(np.float16).view(np.uint8)
        for i in range(4):
            pool[pages[:, :, 0], head[:, :, 0], o + i] = raw[..., i]


def int4_load(pool: np.ndarray, pages, slots, which: int, d: int, ng_k: int, ng_v: int):
    """(codes [T][n_kv][d], s, z [T][n_kv][groups]) of the tokens at (pages[i], slots[i])."""
    ng = ng_v if which else ng_k
    slots = np.asarray(slots)[:, None]
    at, sh = _nibble(d, which, slots, np.arange(d)[None])
    blocks = pool[np.asarray(pages)]                                     # [T][n_kv][block]
    t, h = blocks.shape[:2]
    codes = (np.take_along_axis(blocks, np.broadcast_to(at[:, None], (t, h, d)), 2) >> sh[:, None]) & 15
    o = _pair(d, ng_k, ng_v, which, slots, np.arange(ng)[None])
    raw = np.stack([np.take_along_axis(blocks, np.broadcast_to((o + i)[:, None], (t, h, ng)), 2) for i in range(4)], -1)
    sz = np.ascontiguousarray(raw).view(np.float16)
    return codes.astype(np.uint8), sz[..., 0], sz[..., 1]


def rope(x, cos_sin, interleaved: bool) -> np.ndarray:
    """x [n][heads][d] with its first rot channels rotated by cos_sin [n][rot] (cosines, then sines); float64."""
    x = np.array(x, dtype=np.float64)
    rot = cos_sin.shape[1]
    if rot == 0:
        return x
    c = cos_sin[:, None, :rot // 2].astype(np.float64)
    s = cos_sin[:, None, rot // 2:].astype(np.float64)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = u * c - v * s, u * s + v * c
    return x


def modified_scores(q, k, first_pos: int, scale: float = 0.0, softcap: float = 0.0, window: int = 0, slope: float = 0.0,
                    causal: bool = True, prefix: int = 0) -> np.ndarray:
    """Scores [n][n_k] of queries q [n][d] at positions first_pos .. over keys at 0 ..; -inf where masked."""
    d = q.shape[1]
    t = q @ k.T * (scale if scale else 1.0 / np.sqrt(d))
    if softcap:
        t = softcap * np.tanh(t / softcap)
    i = first_pos + np.arange(q.shape[0])[:, None]
    j = np.arange(k.shape[0])[None]
    t = t - slope * np.abs(i - j)
    seen = np.ones(t.shape, bool)
    if causal:
        seen &= j <= i
    if window:
        seen &= i - j < window
    return np.where(seen | (j < prefix), t, -np.inf)


def masked_attention(t, v):
    """(softmax(t) v, softmax(t) |v|, log sum exp t); rows with nothing give zeros and -inf."""
    if t.shape[1] == 0:
        return np.zeros((t.shape[0], v.shape[1])), np.zeros((t.shape[0], v.shape[1])), np.full(t.shape[0], -np.inf)
    m = t.max(1, keepdims=True)
    p = np.exp(t - np.where(np.isfinite(m), m, 0.0))
    l = p.sum(1, keepdims=True)
    w = p / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return w @ v, w @ np.abs(v), lse
