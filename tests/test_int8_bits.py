"""The bits that the 8-bit decode keeps on its way to the output: the weights' product with the values' scales in two
fp16 parts (22 bits), and sums of centred codes.  Both show where a request's values cancel, so that the result is far
below its terms and its own rounding hides nothing.

Layers whose blocks are written code by code, one KV head.  A query of 8 in one channel, keys of 2 / 255 steps there:
a score is a single rounding of an fp32 fma.  With t - max >= -16 and |t| <= 8 in log2 units, a weight is off by ln 2 times
(8 + 8 + 16 + 16) 2^-24 (the two scores, their difference, the scale) + 2^-21 (the argument, below 16), and 2^-22 for the
power: 2^-18 of it.  What else there is, per term of sizes s |c - 128| and |zero + 128 s|:
 - the parts: 2^-22;
 - the tensor cores' additions: each of a product's 17 addends cut at 2^-24 of the largest, in each of a warp's steps;
 - the zeros' share and the weights' sum: fp32 additions, 2^-24 each, one for each of a lane's tokens;
 - the warps' and the parts' joins and the quotient: 2^-20.
`model` restates the scan in numpy, and shows that the bounds are not met with one part, or with codes as they are.
"""
import numpy as np
import pytest

import oracle as O

D = (64, 128)


def rows(g, n, d, spread):
    """Keys (codes, scales, zeros) of n tokens: channel 0 spans the range, so that scores differ by up to `spread`."""
    c = np.full((n, 1, d), 128, np.uint8)
    c[:, 0, 0] = 128 + g.integers(-spread, spread + 1, n)
    return c, np.full((n, 1), 2.0 / 255, np.float16), np.full((n, 1), -1.0, np.float16)


def weights(k, d):
    """(softmax weights, the logarithm of their sum, scores) of the query 8 in channel 0."""
    c, s, z = k
    t = 8.0 * O.int8_values(c, s, z)[:, 0, 0] / np.sqrt(d)
    p = np.exp(t - t.max())
    return p / p.sum(), t.max() + np.log(p.sum()), t


def unequal(seed, n, d):
    """Random values of unequal scales, and three tokens that take their mean away, each what the one before left."""
    g = np.random.default_rng(seed)
    k = rows(g, n, d, 120)
    k[0][-3:, 0, 0] = 248
    p, lse, t = weights(k, d)
    c = g.integers(0, 256, (n, 1, d)).astype(np.uint8)
    s = (g.uniform(0.5, 1.0, (n, 1)) / 16).astype(np.float16)
    z = (-128.0 * s.astype(np.float64) + g.normal(size=(n, 1)) / 16).astype(np.float16)
    for i in (n - 3, n - 2, n - 1):
        rest = p[:i] @ O.int8_values(c[:i], s[:i], z[:i])[:, 0]
        c[i], s[i], z[i] = O.int8_quantize(-rest[None] / p[i])
    return k, (c, s, z), p, lse, t


def pairs(seed, n, d):
    """Neighbours c and 256 - c beside the middle code, of one scale and a zero of -128 scales: the mean is 0."""
    g = np.random.default_rng(seed)
    k = rows(g, n, d, 120)
    k[0][1::2] = k[0][0::2]
    p, lse, t = weights(k, d)
    a = g.integers(1, 4, (n // 2, 1, d)) * g.choice([-1, 1], (n // 2, 1, d))
    c = np.empty((n, 1, d), np.uint8)
    c[0::2], c[1::2] = 128 + a, 128 - a
    s = np.repeat((g.uniform(0.5, 1.0, (n // 2, 1)) / 16).astype(np.float16), 2, 0)
    return k, (c, s, (-128.0 * s.astype(np.float64)).astype(np.float16)), p, lse, t


def bound(v, p, steps):
    """(the result, how far the output may be off) of values (codes, scales, zeros), `steps` pages a warp one after another."""
    c, s, z = v[0][:, 0].astype(np.float64), v[1].astype(np.float64), v[2].astype(np.float64)
    centred, mid = s * np.abs(c - 128.0), np.abs(z + 128.0 * s)
    want = p @ (z + s * c)
    # a step's addends: its page's products, and the sum so far, which the neighbours of `pairs` leave at nothing; all
    # warps have len(page) steps together; two products a step where a group has more than 4 heads
    page = np.add.reduceat(p[:, None] * s * (c - 128.0), np.arange(0, len(c), 16), axis=0)
    cut = 2 * 17 * 2.0 ** -24 * (steps * np.abs(page).sum(0) + len(page) * (p[:, None] * centred).max(0))
    terms = p @ (centred + mid)
    near = (2.0 ** -18 + 2.0 ** -22 + 2.0 ** -20) * terms + cut + 2 * steps * 2.0 ** -24 * (p @ mid)
    return want, 2.0 ** -8 * np.abs(want) + near


def model(v, t, parts=2, centred=True):
    """The scan of one warp: fp32 weights, fp16 parts, 24-bit sums cut off after every page."""
    c, s, z = v[0][:, 0].astype(np.float64), v[1].astype(np.float64), v[2].astype(np.float64)
    x = np.exp2((t - t.max()) * np.log2(np.e) + 7.0).astype(np.float32).astype(np.float64)[:, None]
    unit = 2.0 ** np.ceil(np.log2(s.max()))
    w = x * s / unit
    hi = w.astype(np.float16).astype(np.float64)
    w = hi + (w - hi).astype(np.float16).astype(np.float64) if parts == 2 else hi
    mid = 128.0 if centred else 0.0
    acc = np.zeros(c.shape[1])
    for i in range(0, len(c), 16):
        acc = acc + (w[i:i + 16] * (c[i:i + 16] - mid)).sum(0)
        e = np.exp2(np.floor(np.log2(np.maximum(np.abs(acc), 1e-300))) - 23.0)
        acc = np.trunc(acc / e) * e
    return (acc * unit + (x * (z + mid * s)).sum(0)) / x.sum()


@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n", [45, 300])
def test_the_bound_is_not_met_with_one_part(d, n):
    k, v, p, lse, t = unequal(n + d, n, d)
    want, near = bound(v, p, 2)
    assert (np.abs(model(v, t) - want) <= near).all()
    assert (np.abs(model(v, t, parts=1) - want) > near).mean() > 0.2


@pytest.mark.parametrize("d", D)
def test_the_bound_is_not_met_without_centring(d):
    k, v, p, lse, t = pairs(d, 640, d)                # what one warp of the long requests has
    want, near = bound(v, p, 40)
    assert (np.abs(model(v, t) - want) <= near).all()
    assert (np.abs(model(v, t, centred=False) - want) > 2 * near).mean() > 0.9


def decoded(g, k, v, n, d, hq, batch):
    """Output and logarithm of `batch` requests on the same pages, each of a query of 8 in channel 0."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int8Cache
    pages = -(-n // 16)
    cache = Int8Cache(batch, hq, 1, d, pages, pages)
    table = g.permutation(pages).astype(np.int32)
    pool = np.full((pages, 1, O.int8_block_bytes(d)), 0xFF, np.uint8)
    pos = np.arange(n)
    for which, x in ((0, k), (1, v)):
        O.int8_store_rows(pool, table[pos // 16], pos % 16, which, *x)
    cache.pages.copy_(torch.from_numpy(pool.reshape(-1)))
    cache.page_table.copy_(torch.from_numpy(np.tile(table, (batch, 1))))
    cache.seq_len.fill_(n)
    q = torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 8.0
    out, lse = torch.empty_like(q), torch.empty(batch, hq, dtype=torch.float32, device="cuda")
    desc = cache.desc(n)
    ws = torch.zeros(B.oscar_decode_int8_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    B.oscar_decode_attention_int8(desc, q, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [3, 4, 7, 16])
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n", [45, 300])
def test_decode_keeps_both_parts_of_the_weights(built_lib, d, hq, n):
    k, v, p, lse, t = unequal(n + d, n, d)
    want, near = bound(v, p, 2)
    got, got_lse = decoded(np.random.default_rng(1), k, v, n, d, hq, 2)
    assert (np.abs(got - want) <= near).all(), np.abs((got - want) / near).max()
    assert (np.abs(got_lse - lse) <= 2.0 ** -18 + 2.0 ** -22 * abs(lse)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [4, 8, 16])
@pytest.mark.parametrize("d", D)
def test_decode_sums_centred_codes(built_lib, d, hq):
    n = 4000                                          # 256 such requests: 60 pages a warp one after another at the most
    k, v, p, lse, t = pairs(d, n, d)
    want, near = bound(v, p, 60)
    got, got_lse = decoded(np.random.default_rng(2), k, v, n, d, hq, 256)
    assert (np.abs(got - want) <= near).all(), np.abs((got - want) / near).max()
    # 120 additions of a lane's weights beside a weight's own 2^-18
    assert (np.abs(got_lse - lse) <= 2.0 ** -18 + 120 * 2.0 ** -24 + 2.0 ** -22 * abs(lse)).all()
