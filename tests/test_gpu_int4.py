"""4-bit layers on the GPU against the float64 oracle: rotate and append,
read back, decode attention, and a run of them together.

Tolerances.  Appended rows are compared exactly: the key row is the rounding
of its exact value and the codes follow from it.  q' carries one bf16
rounding (2^-8) of an fp32 sum (2^-22 of its terms).  The decode's output
carries one bf16 rounding of the result (2^-8), and a fp16 rounding of each
weight and of its product with the scale: 2^-10 of p |s c| at most, with
|s c| <= |zero| + |value| <= 2 max |v|.
"""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda(built_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev_bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def angles(n, rot, theta=1e4):
    f = theta ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Layer:
    """A 4-bit layer of requests of the given lengths, its pages shuffled and every unused slot stale (NaN pairs)."""

    def __init__(self, seed, lens, hq, hk, d, gk, gv, fill=True, extra_pages=2, max_pages=None, tau=65504.0):
        import torch
        from bit_rotated_kv_split_gb300.cache import Int4Cache
        self.g = np.random.default_rng(seed)
        self.lens, self.hq, self.hk, self.d = list(lens), hq, hk, d
        self.gk, self.gv, self.ngk, self.ngv = gk, gv, d // gk, d // gv
        pages = [-(-n // 16) for n in lens]
        n_pages = sum(pages) + extra_pages
        self.cache = Int4Cache(len(lens), hq, hk, d, max_pages or max(max(pages), 1), n_pages, quant_group_k=gk,
                               quant_group_v=gv, tau_k=tau, tau_v=tau)
        order = self.g.permutation(n_pages)
        self.table = np.full((len(lens), self.cache.max_pages_per_seq), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.pool = np.full((n_pages, hk, O.int4_block_bytes(d, self.ngk, self.ngv)), 0xFF, np.uint8)
        self.k, self.v = [], []
        if fill:
            for b, n in enumerate(lens):
                k = O.bf16(self.g.standard_normal((n, hk, d)) * np.where(self.g.random((1, hk, d)) < 0.05, 4, 1))
                v = O.bf16(self.g.standard_normal((n, hk, d)) + 0.3)
                self.k.append(self.put(b, np.arange(n), 0, k)), self.v.append(self.put(b, np.arange(n), 1, v))
        self.cache.page_table.copy_(torch.from_numpy(self.table))
        self.cache.seq_len.copy_(i32(lens))
        self.cache.pages.copy_(torch.from_numpy(self.pool.reshape(-1)))
        self.desc = self.cache.desc(max(max(lens), 0))

    def put(self, b, pos, which, rows):
        """Quantises and stores rows [n][hk][d] at positions pos; returns what they stand for."""
        ng = self.ngv if which else self.ngk
        c, s, z = O.int4_quantize(rows, self.d // ng, self.cache.tau_k)
        pos = np.asarray(pos, dtype=np.int64)
        O.int4_store_rows(self.pool, self.table[b, pos // 16], pos % 16, which, c, s, z, self.ngk, self.ngv)
        return O.int4_values(c, s, z)

    def gpu_pool(self):
        return self.cache.pages.cpu().numpy().reshape(self.pool.shape)

    def status(self):
        return int(self.cache.dev_status.item())


APPENDS = [
    # d, hq, hk, gk, gv, rot, interleaved, tokens of each request, tau
    (128, 32, 8, 128, 128, 128, False, [1], 65504.0),
    (128, 8, 2, 32, 64, 128, True, [3, 1, 17], 65504.0),
    (128, 5, 5, 64, 32, 32, False, [33], 2.0),
    (64, 4, 4, 64, 64, 64, False, [7, 16], 65504.0),
    (64, 9, 3, 32, 32, 16, True, [40, 1], 65504.0),
    (64, 1, 1, 64, 32, 0, False, [2], 65504.0),
    (128, 48, 3, 128, 32, 64, False, [150, 31], 65504.0),
]


@pytest.mark.parametrize("d,hq,hk,gk,gv,rot,inter,tokens,tau", APPENDS)
@pytest.mark.parametrize("packed", [True, False])
def test_append_matches_oracle(d, hq, hk, gk, gv, rot, inter, tokens, tau, packed):
    """The new tokens' pages, k' and q'; every other byte of the pool as it was."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    past = [5 * (i + 1) for i in range(len(tokens))]
    L = Layer(d + hq, [p + t for p, t in zip(past, tokens)], hq, hk, d, gk, gv, fill=False, tau=tau)
    n = sum(tokens)
    g = L.g
    req = np.repeat(np.arange(len(tokens)), tokens)
    pos = np.concatenate([np.arange(p, p + t) for p, t in zip(past, tokens)])
    perm = g.permutation(n)
    req, pos = req[perm], pos[perm]
    q, k, v = (O.bf16(g.standard_normal((n, h, d)) * s) for h, s in ((hq, 1.0), (hk, 3.0), (hk, 1.0)))
    v[0, 0] = 0.0                                   # an all-equal group: scale 0
    if packed:                                      # slices of one projection's output
        qkv = dev_bf16(np.concatenate([q, k, v], 1))
        tq, tk, tv = qkv.split([hq, hk, hk], 1)
    else:
        tq, tk, tv = dev_bf16(q), dev_bf16(k), dev_bf16(v)
    cs = angles(int(pos.max()) + 300, rot)
    rope_pos = pos + g.integers(0, 300, n) if not packed else pos
    rope = B.rope_desc(torch.from_numpy(cs).cuda(), rot, inter)
    q_out = torch.full((n, hq, d), -7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((n, hk, d), -7.0, dtype=torch.bfloat16, device="cuda")
    B.oscar_rope_append_int4(L.desc, rope, tq, tk, tv, i32(req), i32(pos), q_out, k_out,
                             rope_pos=None if packed else i32(rope_pos))
    torch.cuda.synchronize()
    assert L.status() == 0
    k_ref = O.bf16(O.rope(k, cs[rope_pos], inter))
    np.testing.assert_array_equal(host(k_out), k_ref)
    q_ref = O.rope(q, cs[rope_pos], inter)
    near = np.abs(q_ref) * HALF_BF16 + 2.0 ** -22 * np.sqrt((q ** 2).sum(-1, keepdims=True))
    assert (np.abs(host(q_out) - q_ref) <= near).all()
    for i in range(n):
        L.put(int(req[i]), [int(pos[i])], 0, k_ref[i:i + 1])
        L.put(int(req[i]), [int(pos[i])], 1, v[i:i + 1])
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


def test_append_without_queries_in_place_and_infinite_rows():
    """q NULL, k rotated in place; a row with infinities and NaN leaves finite pages and no trace elsewhere."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(3, [20], 4, 2, 128, 32, 32, fill=False)
    k, v = (O.bf16(L.g.standard_normal((20, 2, 128))) for _ in range(2))
    tk, tv = dev_bf16(k), dev_bf16(v)
    tv[4, 1, 3], tv[4, 1, 40], tv[4, 1, 70] = float("inf"), float("-inf"), float("nan")
    cs = angles(20, 128)
    B.oscar_rope_append_int4(L.desc, B.rope_desc(torch.from_numpy(cs).cuda(), 128), None, tk, tv, i32([0] * 20),
                             i32(np.arange(20)), None, tk)
    torch.cuda.synchronize()
    k_ref = O.bf16(O.rope(k, cs, False))
    np.testing.assert_array_equal(host(tk), k_ref)
    L.put(0, np.arange(20), 0, k_ref)
    keep = np.arange(20) != 4
    L.put(0, np.arange(20)[keep], 1, v[keep])
    got = L.gpu_pool()
    _, s, z = O.int4_load(got, [L.table[0, 0]], [4], 1, 128, 4, 4)
    assert np.isfinite(s.astype(np.float64)).all() and np.isfinite(z.astype(np.float64)).all()
    v4 = v.copy()
    v4[4, 1, 3], v4[4, 1, 40], v4[4, 1, 70] = 65504.0, -65504.0, -65504.0
    L.put(0, [4], 1, v4[4:5])
    np.testing.assert_array_equal(got, L.pool)


def test_append_skips():
    """Padding rows are passed over silently; every other bad place is skipped whole and reported."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    bad = [  # req, pos, rope row, page id of that place, status
        (-1, 3, 3, None, 0), (-2, 3, 3, None, 2), (2, 3, 3, None, 2), (0, -1, 3, None, 2), (1, 64, 3, None, 2),
        (0, 40, -1, None, 2), (0, 40, 100, None, 2), (1, 50, 3, -1, 1), (1, 50, 3, 99, 1),
    ]
    for b, p, r, page, status in bad:
        L = Layer(9, [64, 64], 8, 2, 64, 32, 64, fill=False)
        if page is not None:
            L.cache.page_table[b, p // 16] = page
        q, k, v = (dev_bf16(L.g.standard_normal((3, h, 64))) for h in (8, 2, 2))
        q_out, k_out = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
        cs = torch.from_numpy(angles(100, 64)).cuda()
        B.oscar_rope_append_int4(L.desc, B.rope_desc(cs, 64), q, k, v, i32([0, b, 1]), i32([0, p, 1]), q_out, k_out,
                                 rope_pos=i32([0, r, 1]))
        torch.cuda.synchronize()
        assert L.status() == status
        assert bool((q_out[1] == 5.0).all()) and bool((k_out[1] == 5.0).all())
        k_ref = O.bf16(O.rope(host(k), angles(100, 64)[[0, 0, 1]], False))
        for i, (rr, pp) in ((0, (0, 0)), (2, (1, 1))):
            L.put(rr, [pp], 0, k_ref[i:i + 1]), L.put(rr, [pp], 1, host(v)[i:i + 1])
        np.testing.assert_array_equal(L.gpu_pool(), L.pool)
        # the read back skips and reports the same places (a rotation row is nothing to it)
        if 0 <= r < 100:
            L.cache.dev_status.zero_()
            ko, vo = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
            B.oscar_gather_int4(L.desc, i32([0, b, 1]), i32([0, p, 1]), ko, vo)
            torch.cuda.synchronize()
            assert L.status() == status
            assert bool((ko[1] == 5.0).all()) and bool((vo[1] == 5.0).all()) and not bool((ko[0] == 5.0).all())


@pytest.mark.parametrize("d,hk,gk,gv", [(128, 8, 128, 128), (128, 3, 32, 64), (64, 5, 64, 32), (64, 1, 32, 64)])
def test_gather_matches_oracle(d, hk, gk, gv):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(d + hk, [70, 1, 33], hk, hk, d, gk, gv)
    n = 90
    req = L.g.choice(3, n)
    pos = np.array([L.g.integers(0, L.lens[r]) for r in req])
    both = torch.full((n, 2 * hk, d), 9.0, dtype=torch.bfloat16, device="cuda")   # K and V rows side by side
    B.oscar_gather_int4(L.desc, i32(req), i32(pos), both[:, :hk], both[:, hk:])
    torch.cuda.synchronize()
    for at, src in ((slice(0, hk), L.k), (slice(hk, None), L.v)):
        ref = np.stack([O.bf16(src[r][p]) for r, p in zip(req, pos)])
        np.testing.assert_array_equal(host(both[:, at]), ref)
    assert L.status() == 0


def test_many_rows_appended_and_read_back():
    """Enough rows that a warp takes whole tokens, several of them when they are read back; some rows are padding, some
    name bad places, and the last warp's are not all there."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, hq, hk, d = 15_011, 3, 3, 64
    L = Layer(77, [n], hq, hk, d, 32, 64, fill=False)
    q, k, v = (O.bf16(L.g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    cs = angles(n, d)
    req, pos = np.zeros(n, np.int64), L.g.permutation(n)
    req[::7], pos[5::1000], req[11::1001] = -1, -3, 1
    good = (req == 0) & (pos >= 0)
    q_out, k_out = (torch.full((n, h, d), 5.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    B.oscar_rope_append_int4(L.desc, B.rope_desc(torch.from_numpy(cs).cuda(), d), dev_bf16(q), dev_bf16(k), dev_bf16(v),
                             i32(req), i32(pos), q_out, k_out)
    torch.cuda.synchronize()
    assert L.status() == 2
    k_ref = O.bf16(O.rope(k[good], cs[pos[good]], False))
    np.testing.assert_array_equal(host(k_out)[good], k_ref)
    assert (host(k_out)[~good] == 5.0).all() and (host(q_out)[~good] == 5.0).all()
    kc, vc = L.put(0, pos[good], 0, k_ref), L.put(0, pos[good], 1, v[good])
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)
    ko, vo = (torch.full((n, hk, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.oscar_gather_int4(L.desc, i32(req), i32(pos), ko, vo)
    for got, ref in ((host(ko), kc), (host(vo), vc)):
        np.testing.assert_array_equal(got[good], O.bf16(ref))
        assert (got[~good] == 5.0).all()


def decode_ref(L, q, **mods):
    """(attention, its error bound) of q [B][hq][d] over what the cache stands for."""
    slopes = mods.pop("slopes", None)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(L.lens):
        for h in range(L.hq):
            kv = h // (L.hq // L.hk)
            t = O.modified_scores(q[b, h:h + 1], L.k[b][:, kv], n - 1, slope=0.0 if slopes is None else float(slopes[h]), **mods)
            v = L.v[b][:, kv]
            r, _, _ = O.masked_attention(t, v)
            top = np.abs(v).max() * 2 if n else 0.0      # |s c| <= |zero| + |value| <= 2 max|v|
            out[b, h] = r[0]
            bound[b, h] = np.abs(r[0]) * HALF_BF16 + 2.0 ** -10 * top
    return out, bound


def run_decode(L, q, score=None, ws=None, desc=None):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    desc = desc or L.desc
    if ws is None:
        ws = torch.zeros(B.oscar_decode_int4_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    out = torch.full((L.cache.batch, L.hq, L.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.oscar_decode_attention_int4(desc, q, out, ws, score=score)
    torch.cuda.synchronize()
    return out


DECODES = [
    # lens, hq, hk, d, gk, gv, mods
    ([1, 0, 15, 16, 17], 8, 2, 128, 128, 128, {}),
    ([777], 32, 8, 128, 128, 128, {}),
    ([2300, 1, 640], 8, 1, 128, 32, 64, dict(softcap=5.0)),
    ([100, 33], 5, 1, 64, 32, 64, dict(window=40)),
    ([257, 4000], 16, 1, 64, 64, 32, dict(window=1)),
    ([900, 90], 12, 4, 128, 64, 128, dict(slopes=True)),
    ([513, 31], 2, 2, 64, 64, 64, dict(scale=0.5, softcap=20.0, window=300, slopes=True)),
    ([1200], 22, 2, 128, 32, 32, dict(slopes=True, window=700)),
    ([64] * 40, 3, 1, 128, 128, 32, {}),
    ([5000], 9, 1, 64, 32, 32, {}),
]


@pytest.mark.parametrize("lens,hq,hk,d,gk,gv,mods", DECODES)
def test_decode_matches_oracle(lens, hq, hk, d, gk, gv, mods):
    """Unused slots of the last pages hold NaN pairs; the workspace serves twice, bit for bit."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(sum(lens) + hq, lens, hq, hk, d, gk, gv)
    mods = dict(mods)
    q = O.bf16(L.g.standard_normal((len(lens), hq, d)))
    rows = torch.zeros(len(lens), hq + 3, d, dtype=torch.bfloat16, device="cuda")
    rows[:, :hq] = dev_bf16(q)
    sl = None
    if mods.get("slopes"):
        mods["slopes"] = np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
        sl = torch.from_numpy(mods["slopes"]).cuda()
    score = B.score_desc(mods.get("scale", 0.0), mods.get("softcap", 0.0), mods.get("window", 0), sl)
    ws = torch.zeros(B.oscar_decode_int4_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda")
    out = run_decode(L, rows[:, :hq], score, ws)
    again = run_decode(L, rows[:, :hq], score, ws)
    ref, bound = decode_ref(L, q, **mods)
    err = np.abs(host(out) - ref)
    assert (err <= bound).all(), "worst %.3g of its bound" % np.nanmax(err / np.maximum(bound, 1e-30))
    assert bool((out.view(torch.int16) == again.view(torch.int16)).all())
    assert L.status() == 0


RAGGED = [
    # lens of many requests: runs that are whole, split over several CTAs, empty, of one token
    ([0, 3, 0, 0, 17] * 60 + [900, 0, 1, 2100, 64, 65], 2, 1, 64, 64, 32, {}),          # more requests than threads
    ([9000, 5, 0, 7000, 1025, 1024, 1023, 1039, 2], 4, 2, 64, 32, 64, {}),
    ([30000, 1, 12000], 12, 1, 64, 64, 64, dict(softcap=9.0)),                           # two head sets
    ([40000], 8, 8, 64, 64, 64, dict(window=20001)),
    ([6000, 6000, 6001, 5999, 1, 6000], 8, 2, 128, 128, 64, dict(window=1500, slopes=True)),
]


@pytest.mark.parametrize("lens,hq,hk,d,gk,gv,mods", RAGGED)
def test_decode_ragged_batches(lens, hq, hk, d, gk, gv, mods):
    test_decode_matches_oracle(lens, hq, hk, d, gk, gv, mods)


def test_workspace_shared_by_calls_of_different_sizes():
    """One workspace for layers and batches of all sizes, one call after the other (it is zero-filled once)."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    shapes = [([5000, 300], 8, 2, 128, 128, 128), ([1] * 400, 2, 1, 64, 64, 64), ([2500] * 9, 16, 2, 128, 32, 64),
              ([20000], 4, 1, 64, 32, 32), ([3000, 0, 700], 24, 8, 128, 64, 128)]
    Ls = [Layer(60 + i, *s) for i, s in enumerate(shapes)]
    ws = torch.zeros(max(B.oscar_decode_int4_workspace_bytes(L.desc) for L in Ls), dtype=torch.uint8, device="cuda")
    qs = [O.bf16(L.g.standard_normal((len(L.lens), L.hq, L.d))) for L in Ls]
    for L, q in list(zip(Ls, qs)) * 2:
        ref, bound = decode_ref(L, q)
        assert (np.abs(host(run_decode(L, dev_bf16(q), ws=ws)) - ref) <= bound).all()


def test_decode_peaked_and_far_scores():
    """One key far above the rest, scores of hundreds: the output is that key's value."""
    import torch
    L = Layer(5, [1500, 300], 8, 2, 128, 32, 32)
    q = np.zeros((2, 8, 128))
    for b, j in ((0, 1490), (1, 7)):
        for h in range(8):
            q[b, h] = O.bf16(L.k[b][j, h // 4] * 30)
    out = host(run_decode(L, dev_bf16(q)))
    ref, bound = decode_ref(L, q)
    assert (np.abs(out - ref) <= bound).all()
    torch.cuda.synchronize()


def test_decode_query_of_zeros_and_of_extreme_size():
    """A zero query takes the mean; queries of 2^-100 and 2^20 are scaled exactly."""
    import torch
    L = Layer(6, [1000, 40], 4, 1, 64, 64, 32)
    q = np.zeros((2, 4, 64))
    q[:, 1] = O.bf16(L.g.standard_normal((2, 64))) * 2.0 ** -100
    q[:, 2] = O.bf16(L.g.standard_normal((2, 64))) * 2.0 ** 12
    q[:, 3] = O.bf16(L.g.standard_normal((2, 64)) * 2.0 ** L.g.integers(-30, 1, 64))
    out = host(run_decode(L, dev_bf16(q)))
    ref, bound = decode_ref(L, q)
    # scores of up to 2^17 in fp32 are off by up to 2^-6, so only the head's own largest key counts for head 2
    for b in range(2):
        t = O.modified_scores(q[b, 2:3], L.k[b][:, 0], L.lens[b] - 1)[0]
        top = np.sort(t)[-2:]
        if top[1] - top[0] < 8:
            bound[b, 2] = np.inf
    assert (np.abs(out - ref) <= bound).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,softcap", [([300, 40, 5000], 0.0), ([20000, 1], 7.0)])
def test_decode_query_with_nan_shows_and_stays_alone(lens, softcap):
    """A NaN in a head's query makes that head's result NaN, its request's pages split or not, and no other's."""
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(77, lens, 6, 2, 64, 64, 64)
    q = O.bf16(L.g.standard_normal((len(lens), 6, 64)))
    ref, bound = decode_ref(L, q, softcap=softcap)
    for b in range(len(lens)):
        bad = dev_bf16(q)
        bad[b, 4, 9] = float("nan")
        out = host(run_decode(L, bad, B.score_desc(0.0, softcap, 0, None)))
        assert np.isnan(out[b, 4]).all()
        out[b, 4] = ref[b, 4]
        assert (np.abs(out - ref) <= bound).all()


@pytest.mark.parametrize("kscale,vscale", [(1e-3, 1e-4), (100.0, 3000.0)])
def test_decode_small_and_large_values(kscale, vscale):
    """Scales near fp16's ends: keys and values far from 1, and a token with one large channel among small ones."""
    import torch
    L = Layer(8, [700], 4, 1, 128, 64, 64)
    k = O.bf16(L.g.standard_normal((700, 1, 128)) * kscale)
    v = O.bf16(L.g.standard_normal((700, 1, 128)) * vscale * np.exp(L.g.standard_normal((700, 1, 1)) * 2))
    L.k[0], L.v[0] = L.put(0, np.arange(700), 0, k), L.put(0, np.arange(700), 1, v)
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    q = O.bf16(L.g.standard_normal((1, 4, 128)) / kscale)
    out = host(run_decode(L, dev_bf16(q)))
    ref, bound = decode_ref(L, q)
    assert (np.abs(out - ref) <= bound).all()


def test_decode_reports_and_survives_bad_lengths_and_pages():
    import torch
    L = Layer(11, [200, 50, 90], 8, 2, 128, 128, 128)
    q = O.bf16(L.g.standard_normal((3, 8, 128)))
    desc = L.cache.desc(120)                        # request 0 is longer than the bound: clamped
    out = host(run_decode(L, dev_bf16(q), desc=desc))
    assert L.status() == 2
    M = Layer(11, [200, 50, 90], 8, 2, 128, 128, 128)
    M.cache.seq_len.copy_(i32([120, 50, -4]))       # -4 counts as none
    got = host(run_decode(M, dev_bf16(q)))
    assert M.status() == 2
    np.testing.assert_array_equal(out[:2], got[:2])
    assert (got[2] == 0).all()
    M.cache.dev_status.zero_()
    M.cache.seq_len.copy_(i32([200, 50, 90]))
    M.cache.page_table[1, 1] = 1000                 # tokens 16 .. 31 of request 1 are passed over
    got = host(run_decode(M, dev_bf16(q)))
    assert M.status() == 1
    keep = np.r_[0:16, 32:50]
    M.lens = [200, 34, 90]
    M.k[1], M.v[1] = M.k[1][keep], M.v[1][keep]
    ref, bound = decode_ref(M, q)
    assert (np.abs(got - ref) <= bound).all()


def test_offsets_past_32_bits():
    """Pages at the far end of a pool of over 4 GB: append, read back, decode."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    n_pages = 260_000
    cache = Int4Cache(1, 32, 8, 128, 4, n_pages)
    assert cache.pages.numel() > 1 << 32
    cache.page_table.copy_(i32([[n_pages - 1, n_pages - 9, 3, n_pages - 4]]))
    cache.seq_len.fill_(60)
    g = np.random.default_rng(1)
    k, v = (O.bf16(g.standard_normal((60, 8, 128))) for _ in range(2))
    desc = cache.desc(64)
    req, pos = i32([0] * 60), i32(np.arange(60))
    B.oscar_rope_append_int4(desc, None, None, dev_bf16(k), dev_bf16(v), req, pos, None)
    ko, vo = (torch.empty(60, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.oscar_gather_int4(desc, req, pos, ko, vo)
    kc, vc = (O.int4_values(*O.int4_quantize(x, 128, 65504.0)) for x in (k, v))
    np.testing.assert_array_equal(host(ko), O.bf16(kc))
    np.testing.assert_array_equal(host(vo), O.bf16(vc))
    q = O.bf16(g.standard_normal((1, 32, 128)))
    ws = torch.zeros(B.oscar_decode_int4_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 32, 128, dtype=torch.bfloat16, device="cuda")
    B.oscar_decode_attention_int4(desc, dev_bf16(q), out, ws)

    class L:
        lens, hq, hk = [60], 32, 8
    L.k, L.v = [kc], [vc]
    ref, bound = decode_ref(L, q)
    assert (np.abs(host(out) - ref) <= bound).all()
    assert int(cache.dev_status.item()) == 0


def test_layer_run_prompt_then_tokens():
    """As a serving program has them: a prompt is rotated, appended and attended; then tokens are appended and decoded in
    a captured graph, replayed step by step on a stream of its own.  Each step's output is that of the oracle over
    what the cache stands for, and the rows read back are the cache's."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    hq, hk, d, n0, steps = 8, 2, 128, 45, 5
    L = Layer(21, [n0 + steps], hq, hk, d, 64, 32, fill=False)
    g, n = L.g, n0 + steps
    q, k, v = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    cs = angles(n, d, 1e6)
    rope = B.rope_desc(torch.from_numpy(cs).cuda(), d)
    score = B.score_desc(softcap=30.0)
    kr = O.bf16(O.rope(k, cs, False))
    # the prompt
    tq, tk, tv = dev_bf16(q[:n0]), dev_bf16(k[:n0]), dev_bf16(v[:n0])
    q_rot, k_rot = torch.empty_like(tq), torch.empty_like(tk)
    B.oscar_rope_append_int4(L.desc, rope, tq, tk, tv, i32([0] * n0), i32(np.arange(n0)), q_rot, k_rot)
    pd = B.prompt_desc(1, hq, hk, d, n0, n0, n0, n0)
    cu, pws = i32([0, n0]), torch.zeros(B.oscar_prompt_workspace_bytes(pd), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q_rot)
    B.oscar_prompt_attention(pd, q_rot, k_rot, tv, cu, cu, out, pws, score=score)
    got = host(out)
    for h in range(hq):
        t = O.modified_scores(host(q_rot)[:, h], kr[:n0, h // 4], 0, softcap=30.0)
        r, r_abs, _ = O.masked_attention(t, v[:n0, h // 4])
        assert (np.abs(got[:, h] - r) <= HALF_BF16 * (np.abs(r) + r_abs) + 2.0 ** -14).all()
    # the tokens
    seq = L.cache.seq_len
    seq.fill_(n0)
    sq, sk, sv = (torch.zeros(1, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hk, hk))
    pos, req = i32([n0]), i32([0])
    q1, o1 = torch.empty_like(sq), torch.empty_like(sq)
    ws = torch.zeros(B.oscar_decode_int4_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda")

    def step():
        seq.add_(1)
        B.oscar_rope_append_int4(L.desc, rope, sq, sk, sv, req, pos, q1)
        B.oscar_decode_attention_int4(L.desc, q1, o1, ws, score=score)
        pos.add_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for i in range(n0, n):
            sq.copy_(dev_bf16(q[i:i + 1])), sk.copy_(dev_bf16(k[i:i + 1])), sv.copy_(dev_bf16(v[i:i + 1]))
            graph.replay()
            side.synchronize()
            L.lens = [i + 1]
            L.k = [O.int4_values(*O.int4_quantize(kr[:i + 1], 64, 65504.0))]
            L.v = [O.int4_values(*O.int4_quantize(v[:i + 1], 32, 65504.0))]
            ref, bound = decode_ref(L, host(q1), softcap=30.0)
            assert (np.abs(host(o1) - ref) <= bound).all()
    ko, vo = (torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.oscar_gather_int4(L.desc, i32([0] * n), i32(np.arange(n)), ko, vo)
    np.testing.assert_array_equal(host(ko), O.bf16(L.k[0]))
    np.testing.assert_array_equal(host(vo), O.bf16(L.v[0]))
    assert L.status() == 0


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured decodes replayed at once on two streams, each with its workspace, give the eager results."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    Ls = [Layer(31 + i, [3000, 777], 8, 2, 128, 128, 128) for i in range(2)]
    qs = [dev_bf16(L.g.standard_normal((2, 8, 128))) for L in Ls]
    want = [run_decode(L, q) for L, q in zip(Ls, qs)]
    graphs, outs, keep = [], [], []
    for L, q in zip(Ls, qs):
        ws = torch.zeros(B.oscar_decode_int4_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.oscar_decode_attention_int4(L.desc, q, out, ws)
        graphs.append(graph), outs.append(out), keep.append(ws)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert bool((a.view(torch.int16) == b.view(torch.int16)).all())


def weighted_ref(L, q, **mods):
    """(attention, its error bound) of q over what the cache stands for, each key's error counted with its weight.

    A weight p (the largest of a row 1, their sum at least 1) is rounded to fp16 for the sums of zeros and weights, and
    its product with the scale s once more: 2^-11 of p |v - out| and of p |s c|.  Below fp16's normal range (weights
    are held times 2^7 or more, products times 2^-ve with s 2^-ve >= 2^-14) the steps are 2^-32 of a weight, and 2^-17
    of s c.  fp32 sums, products and powers: 2^-13 of all terms.  The result is rounded to bf16.
    """
    slopes = mods.pop("slopes", None)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(L.lens):
        if n == 0:
            continue
        pos = np.arange(n)
        c, s, z = O.int4_load(L.pool, L.table[b, pos // 16], pos % 16, 1, L.d, L.ngk, L.ngv)
        sc = np.repeat(s.astype(np.float64), L.d // L.ngv, -1) * c
        z = np.repeat(z.astype(np.float64), L.d // L.ngv, -1)
        for h in range(L.hq):
            kv = h // (L.hq // L.hk)
            t = O.modified_scores(q[b, h:h + 1], L.k[b][:, kv], n - 1, slope=0.0 if slopes is None else float(slopes[h]), **mods)[0]
            seen = np.isfinite(t)
            p = np.exp(t[seen] - t[seen].max())
            zv, sv = z[seen, kv], sc[seen, kv]
            v = zv + sv
            r = p @ v / p.sum()
            away = np.abs(v - r)
            near = 2.0 ** -11 * (p @ away + p @ sv) + 2.0 ** -13 * (p @ (np.abs(zv) + sv + away))
            near += np.minimum(p, 2.0 ** -32) @ away + np.minimum(p, 2.0 ** -17) @ sv
            out[b, h], bound[b, h] = r, np.abs(r) * HALF_BF16 + near / p.sum()
    return out, bound


@pytest.mark.parametrize("softcap", [1e3, 1e5, 1e7, 1e12, 1e30, 1e38])
@pytest.mark.parametrize("d,slopes", [(128, False), (64, True)])
def test_decode_large_caps_leave_ordinary_scores(softcap, d, slopes):
    """Scores of ordinary size under a cap far above them: the cap's error is one of the score, not of the cap."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(91, [2000, 40, 3000], 8, 2, d, 64, 32)
    q = O.bf16(L.g.standard_normal((3, 8, d)))
    mods = dict(softcap=softcap)
    sl = None
    if slopes:
        mods["slopes"] = np.exp2(-8.0 * np.arange(1, 9) / 8).astype(np.float32)
        sl = torch.from_numpy(mods["slopes"]).cuda()
    out = host(run_decode(L, dev_bf16(q), B.score_desc(0.0, softcap, 0, sl)))
    ref, bound = weighted_ref(L, q, **mods)
    assert (np.abs(out - ref) <= bound).all(), "worst %.3g of its bound" % np.nanmax(np.abs(out - ref) / bound)


def test_decode_cap_of_scores_on_both_sides_of_it():
    """Scores from a hundredth of the cap to a hundred times it in one request, small and large in the same warp."""
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(92, [700, 90], 4, 1, 128, 128, 128)
    q = O.bf16(L.g.standard_normal((2, 4, 128)) * np.array([0.01, 0.3, 3.0, 60.0])[None, :, None])
    for softcap in (1.0, 8.0, 300.0):
        out = host(run_decode(L, dev_bf16(q), B.score_desc(0.0, softcap, 0, None)))
        ref, bound = weighted_ref(L, q, softcap=softcap)
        assert (np.abs(out - ref) <= bound).all()




@pytest.mark.parametrize("gk,gv,big,lens,hq,d,mods", [
    (128, 128, 3.0, [900, 2500], 4, 128, {}),
    (32, 32, 300.0, [900, 2500], 4, 128, {}),
    (64, 64, 6e4, [900, 2500], 12, 128, {}),
    (32, 64, 6e4, [3, 17, 1100], 5, 64, dict(softcap=100.0)),
    (128, 32, 6e4, [2500], 8, 128, dict(window=2000, slopes=True)),
    (64, 32, 6e4, [9000, 33, 0, 5000], 9, 64, {}),             # split over CTAs
])
def test_decode_large_value_of_no_weight_leaves_small_ones(gk, gv, big, lens, hq, d, mods):
    """One token's values far above all others': a head that gives it no weight keeps its precision, one that gives it all
    takes it."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(93, lens, hq, 1, d, gk, gv, fill=False)
    q = np.zeros((len(lens), hq, d))
    for b, n in enumerate(L.lens):
        k = O.bf16(L.g.standard_normal((n, 1, d)))
        v = O.bf16(L.g.standard_normal((n, 1, d)) * 0.003 + 0.01)
        if n:
            k[n // 3, 0, 5] = 64.0
            v[n // 3] = O.bf16(L.g.standard_normal((1, d)).clip(-1, 1) * big)
        L.k.append(L.put(b, np.arange(n), 0, k)), L.v.append(L.put(b, np.arange(n), 1, v))
        q[b] = O.bf16(L.g.standard_normal((hq, d)) * 0.1)
        q[b, :, 5] = np.resize([-16.0, 16.0, -20.0, 0.5], hq)
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    mods, sl = dict(mods), None
    if mods.get("slopes"):
        mods["slopes"] = np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
        sl = torch.from_numpy(mods["slopes"]).cuda()
    out = host(run_decode(L, dev_bf16(q), B.score_desc(0.0, mods.get("softcap", 0.0), mods.get("window", 0), sl)))
    ref, bound = weighted_ref(L, q, **mods)
    err = np.abs(out - ref)
    assert (err <= bound).all(), "worst %.3g of its bound" % np.nanmax(err / np.maximum(bound, 1e-30))
    assert L.status() == 0


def test_decode_large_value_among_small_ones_on_bad_pages():
    """The same where a page is not in the pool: it is passed over and reported."""
    import torch
    L = Layer(98, [200, 50], 6, 2, 128, 64, 32, fill=False)
    for b, n in enumerate(L.lens):
        k, v = O.bf16(L.g.standard_normal((n, 2, 128))), O.bf16(L.g.standard_normal((n, 2, 128)) * 0.003 + 0.01)
        k[5, :, 5], v[5] = 64.0, 5e4
        v[5, :, ::2] = -5e4
        L.k.append(L.put(b, np.arange(n), 0, k)), L.v.append(L.put(b, np.arange(n), 1, v))
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    L.cache.page_table[1, 1] = 1000                 # tokens 16 .. 31 of request 1 are passed over
    q = O.bf16(L.g.standard_normal((2, 6, 128)) * 0.1)
    q[:, :, 5] = -20.0
    out = host(run_decode(L, dev_bf16(q)))
    assert L.status() == 1
    keep = np.r_[0:16, 32:50]
    L.lens, L.k[1] = [200, 34], L.k[1][keep]
    first, second = L.table[1, 0], L.table[1, 2]    # tokens 32 .. 49 as 16 .. 33
    L.table[1, 1], L.table[1, 2], L.table[1, 0] = second, L.table[1, 3], first
    ref, bound = weighted_ref(L, q)
    assert (np.abs(out - ref) <= bound).all()


@pytest.mark.parametrize("spread", [4, 12, 20])
def test_decode_values_of_all_sizes(spread):
    """Tokens and groups of values from 2^-spread to 2^13 (scales down into fp16's subnormal range, some 0)."""
    import torch
    L = Layer(94, [1300, 33], 6, 2, 128, 64, 32, fill=False)
    for b, n in enumerate(L.lens):
        k = O.bf16(L.g.standard_normal((n, 2, 128)))
        v = O.bf16(L.g.standard_normal((n, 2, 128)) * 2.0 ** L.g.integers(-spread, 14, (n, 2, 1)) *
                   np.repeat(2.0 ** -L.g.integers(0, 5, (n, 2, 4)) * (L.g.random((n, 2, 4)) < 0.9), 32, -1))
        L.k.append(L.put(b, np.arange(n), 0, k)), L.v.append(L.put(b, np.arange(n), 1, v))
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    q = O.bf16(L.g.standard_normal((2, 6, 128)))
    out = host(run_decode(L, dev_bf16(q)))
    ref, bound = weighted_ref(L, q)
    assert (np.abs(out - ref) <= bound).all(), "worst %.3g of its bound" % np.nanmax(np.abs(out - ref) / bound)


@pytest.mark.parametrize("lens,hq,hk,d,gk,gv,window", [
    ([777, 64, 65, 1024, 1025], 4, 2, 64, 64, 64, 0),
    ([5000], 9, 1, 64, 32, 32, 0),
    ([9000, 5, 0, 7000, 1025, 1024, 1023, 1039, 2], 4, 2, 64, 32, 64, 0),
    ([30000, 1, 12000], 12, 1, 128, 64, 64, 0),
    ([40000], 8, 8, 128, 128, 128, 20001),
    ([0, 3, 0, 0, 17] * 60 + [900, 0, 1, 2100, 64, 65], 2, 1, 64, 64, 32, 0),
    ([6000, 6000, 6001, 5999, 1, 6000], 8, 2, 128, 128, 64, 1500),
    ([2000] * 33, 2, 2, 64, 64, 64, 0),
])
def test_decode_counts_each_page_once(lens, hq, hk, d, gk, gv, window):
    """Equal weights, and values that are 1 in one channel for the pages of one remainder mod d: a page left out or taken
    twice, at the ends of a run or of a CTA's share or within them, moves that channel by several times its bound."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(sum(lens) + d, lens, hq, hk, d, gk, gv, fill=False)
    for b, n in enumerate(lens):
        v = np.zeros((n, hk, d))
        v[np.arange(n), :, np.arange(n) // 16 % d] = 1.0
        L.k.append(L.put(b, np.arange(n), 0, O.bf16(L.g.standard_normal((n, hk, d))))), L.v.append(L.put(b, np.arange(n), 1, v))
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    q = np.zeros((len(lens), hq, d))
    out = host(run_decode(L, dev_bf16(q), B.score_desc(0.0, 0.0, window, None)))
    ref, bound = weighted_ref(L, q, window=window)
    assert (np.abs(out - ref) <= bound).all(), "worst %.3g of its bound" % np.nanmax(np.abs(out - ref) / np.maximum(bound, 1e-30))
    for b, n in enumerate(lens):
        if n > 16:
            assert bound[b].max() < 0.5 * 16 / min(n, window or n)


@pytest.mark.parametrize("lens", [[1000, 40], [6000, 3]])
def test_decode_queries_of_all_sizes_with_keys_apart(lens):
    """Queries of 2^-100 to 2^16 with, for each head, one key whose score is several times all others': the small ones take
    the mean, the large ones that key's value, each within the weighted bound."""
    import torch
    L = Layer(99, lens, 4, 1, 64, 64, 32, fill=False)
    sizes = 2.0 ** np.array([-100.0, 3.0, 12.0, 16.0])
    q = np.zeros((len(lens), 4, 64))
    for b, n in enumerate(lens):
        unit = O.bf16(L.g.standard_normal((4, 64)))
        k, v = O.bf16(L.g.standard_normal((n, 1, 64))), O.bf16(L.g.standard_normal((n, 1, 64)))
        for h in range(4):
            k[(h + 1) * n // 5, 0] = 4.0 * np.sign(unit[h])
        L.k.append(L.put(b, np.arange(n), 0, k)), L.v.append(L.put(b, np.arange(n), 1, v))
        q[b] = unit * sizes[:, None]
    L.cache.pages.copy_(torch.from_numpy(L.pool.reshape(-1)))
    out = host(run_decode(L, dev_bf16(q)))
    ref, bound = weighted_ref(L, q)
    assert (np.abs(out - ref) <= bound).all(), "worst %.3g of its bound" % np.nanmax(np.abs(out - ref) / bound)
    for b, n in enumerate(lens):
        if n > 4:
            for h in (2, 3):
                np.testing.assert_allclose(out[b, h], L.v[b][(h + 1) * n // 5, 0], rtol=2.0 ** -8 + 2.0 ** -10, atol=2.0 ** -9)


@pytest.mark.parametrize("lens,hq,hk,d,gk,gv,mods", RAGGED + DECODES)
def test_decode_within_the_weighted_bound(lens, hq, hk, d, gk, gv, mods):
    """The batches above with each key's error counted with its weight, which for long requests is a small part of what the
    largest value would allow."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(sum(lens) + hq, lens, hq, hk, d, gk, gv)
    mods, sl = dict(mods), None
    if mods.get("slopes"):
        mods["slopes"] = np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
        sl = torch.from_numpy(mods["slopes"]).cuda()
    q = O.bf16(L.g.standard_normal((len(lens), hq, d)))
    score = B.score_desc(mods.get("scale", 0.0), mods.get("softcap", 0.0), mods.get("window", 0), sl)
    out = host(run_decode(L, dev_bf16(q), score))
    ref, bound = weighted_ref(L, q, **mods)
    assert (np.abs(out - ref) <= bound).all(), "worst %.3g of its bound" % np.nanmax(np.abs(out - ref) / np.maximum(bound, 1e-30))


def test_append_codes_where_differences_need_more_than_fp32():
    """Quotients next to a half, on the side that a difference rounded to fp32 loses: a zero 2^-25 of the values beside it."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, hk, d = 60, 2, 64
    L = Layer(95, [n], hk, hk, d, 32, 64, fill=False)
    g = L.g
    v = np.zeros((n, hk, d))
    for i in range(n):
        s = 2.0 ** int(g.integers(-6, 4))                       # every group: 15 s at most, halves of s, the least 2^-24 ..
        for h in range(hk):
            x = (g.integers(0, 31, d) * 0.5) * s
            x[::32] = 15.0 * s
            x[7::32] = 2.0 ** float(g.integers(-40, -20)) * (1 if g.random() < 0.5 else -1)
            v[i, h] = np.where(x == 0, s, x)
    v = O.bf16(v)
    k = O.bf16(v[::-1] * 1.0)
    B.oscar_rope_append_int4(L.desc, None, None, dev_bf16(k), dev_bf16(v), i32([0] * n), i32(np.arange(n)), None)
    torch.cuda.synchronize()
    L.put(0, np.arange(n), 0, k), L.put(0, np.arange(n), 1, v)
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


def test_append_scales_where_the_range_needs_more_than_fp32():
    """Ranges of 15 (2 m + 1) 2^-25, halfway between two subnormal scales, less or more by a least value of 2^-50."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, d = 40, 64
    L = Layer(96, [n], 1, 1, d, 64, 64, fill=False)
    v = np.zeros((n, 1, d))
    for i in range(n):
        m = i % 8
        v[i, 0] = 15.0 * (2 * m + 1) * 2.0 ** -25 * (np.arange(d) % 4) / 4 + 2.0 ** -30
        v[i, 0, 3] = 15.0 * (2 * m + 1) * 2.0 ** -25
        v[i, 0, 8] = (1.0, -1.0)[i // 8 % 2] * 2.0 ** -(50 + i % 3)
        if i // 16 % 2:
            v[i] = -v[i]
    v = O.bf16(v)
    B.oscar_rope_append_int4(L.desc, None, None, dev_bf16(v), dev_bf16(v), i32([0] * n), i32(np.arange(n)), None)
    torch.cuda.synchronize()
    L.put(0, np.arange(n), 0, v), L.put(0, np.arange(n), 1, v)
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


@pytest.mark.parametrize("inter", [False, True])
def test_append_rotates_the_smallest_keys_exactly(inter):
    """Keys at and below fp32's least normal number: k' is the rounding of its exact value there as well."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, d = 3000, 64
    L = Layer(97, [n], 2, 2, d, 64, 64, fill=False)
    k = O.bf16(L.g.standard_normal((n, 2, d)) * 2.0 ** L.g.integers(-132, -118, (n, 2, 1)))
    cs = angles(n, d)
    tk = dev_bf16(k)
    np.testing.assert_array_equal(host(tk), k)
    B.oscar_rope_append_int4(L.desc, B.rope_desc(torch.from_numpy(cs).cuda(), d, inter), None, tk, tk.clone(), i32([0] * n),
                             i32(np.arange(n)), None, tk)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(tk), O.bf16(O.rope(k, cs, inter)))
