"""Prompt attention on the GPU against the float64 oracle.

Tolerance: one bf16 rounding of the result (2^-8 of it), one of each weight
(2^-8 of sum p |v|), and fp32 scores (2^-14 covers |t| up to some hundreds).
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


def run(case_seed, nq, nk, hq, hk, d, causal=True, prefix=None, gap=0, packed=False, slack=1, **mods):
    """One call over requests of nq[i] queries and nk[i] keys; `gap` rows of NaN keys and values (and untouched query
    rows) before the first and after the last request; `slack` times the longest request as bounds.  Returns (out,
    lse) after checking them."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(case_seed)
    tq, tk = sum(nq) + 2 * gap, sum(nk) + 2 * gap
    q, k, v = O.bf16(g.standard_normal((tq, hq, d))), O.bf16(g.standard_normal((tk, hk, d))), O.bf16(g.standard_normal((tk, hk, d)) + 0.2)
    cu_q, cu_k = gap + np.r_[0, np.cumsum(nq)], gap + np.r_[0, np.cumsum(nk)]
    dq, dk, dv = dev_bf16(q), dev_bf16(k), dev_bf16(v)
    if gap:
        for t in (dk, dv):
            t[:gap], t[tk - gap:] = float("nan"), float("inf")
    if packed:
        both = torch.cat([dq, dk, dv], 1)
        dq, dk, dv = both.split([hq, hk, hk], 1)
    out = torch.full((tq, hq, d), -3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq, hq), -3.0, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = B.prompt_desc(len(nq), hq, hk, d, slack * max(nq), slack * max(nk), tq, tk, causal, st)
    sl = None
    slopes = np.zeros(hq, np.float32)
    if mods.pop("slopes", False):
        slopes = np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
        sl = torch.from_numpy(slopes).cuda()
    score = B.score_desc(mods.get("scale", 0.0), mods.get("softcap", 0.0), mods.get("window", 0), sl)
    ws = torch.zeros(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    args = (desc, dq, dk, dv, i32(cu_q), i32(cu_k), out, ws)
    kw = dict(score=score, prefix_len=None if prefix is None else i32(prefix), lse=lse)
    B.oscar_prompt_attention(*args, **kw)
    torch.cuda.synchronize()
    first = out.clone()
    B.oscar_prompt_attention(*args, **kw)           # the workspace serves again
    torch.cuda.synchronize()
    assert bool((first.view(torch.int16) == out.view(torch.int16)).all())
    got, got_l = host(out), lse.cpu().numpy().astype(np.float64)
    if gap:
        for t in (got, got_l):
            assert (t[:gap] == -3.0).all() and (t[tq - gap:] == -3.0).all()
    assert int(st.item()) == 0
    for b in range(len(nq)):
        for h in range(hq):
            kb, vb = k[cu_k[b]:cu_k[b + 1], h // (hq // hk)], v[cu_k[b]:cu_k[b + 1], h // (hq // hk)]
            t = O.modified_scores(q[cu_q[b]:cu_q[b + 1], h], kb, nk[b] - nq[b], slope=float(slopes[h]), causal=causal,
                                  prefix=0 if prefix is None else prefix[b], **mods)
            r, r_abs, l = O.masked_attention(t, vb)
            o = got[cu_q[b]:cu_q[b + 1], h]
            err = np.abs(o - r)
            bound = HALF_BF16 * (np.abs(r) + r_abs) + 2.0 ** -14
            assert (err <= bound).all(), "request %d head %d: worst %.3g of its bound" % (b, h, np.nanmax(err / bound))
            gl = got_l[cu_q[b]:cu_q[b + 1], h]
            empty = np.isneginf(l)
            assert np.isneginf(gl[empty]).all() and (o[empty] == 0).all()
            assert np.abs(gl[~empty] - l[~empty]).max(initial=0.0) <= 2.0 ** -14
    return out, lse


CASES = [
    # nq, nk, hq, hk, d, kwargs
    ([1], [1], 1, 1, 128, {}),
    ([300], [300], 4, 1, 128, {}),
    ([129, 5, 128], [129, 5, 128], 8, 2, 64, dict(packed=True)),
    ([64, 0, 33], [64, 17, 33], 6, 2, 128, dict(gap=40)),
    ([7, 20], [700, 20], 8, 1, 128, dict(gap=3)),
    ([50], [20], 4, 4, 64, {}),                                  # the first 30 queries see nothing
    ([50, 9], [0, 0], 4, 2, 128, {}),                            # no key at all
    ([200, 31], [200, 300], 5, 1, 64, dict(window=50, gap=9)),
    ([150], [400], 16, 1, 128, dict(softcap=10.0, window=130)),
    ([260, 100], [260, 100], 3, 3, 128, dict(prefix=[70, 200])),
    ([260], [500], 4, 2, 64, dict(prefix=[130], window=20, softcap=3.0)),
    ([130, 60], [130, 200], 12, 4, 128, dict(causal=False)),
    ([130], [280], 8, 2, 128, dict(causal=False, window=64, slopes=True)),
    ([333], [333], 10, 2, 64, dict(slopes=True)),
    ([96], [1100], 16, 2, 64, dict(slopes=True, softcap=20.0, scale=0.3, prefix=[10], gap=17)),
    ([1], [4000], 32, 8, 128, {}),
    ([24, 2], [3100, 2000], 8, 2, 128, dict(window=1500)),
    ([1000], [1000], 2, 1, 128, {}),
    ([3] * 30, [3] * 30, 4, 1, 64, {}),
    ([257], [257], 7, 1, 128, dict(packed=True)),
    # keys split over several CTAs: alternate tiles for few rows, two row tiles, requests with few keys or none among them
    ([5, 3, 1], [2500, 90, 0], 8, 2, 128, {}),
    ([100, 40], [5000, 1300], 8, 2, 64, dict(gap=5)),
    ([20], [4000], 4, 1, 128, dict(prefix=[700], window=300)),
    ([33, 1], [2049, 2048], 6, 2, 64, dict(softcap=8.0, slopes=True)),
    ([2], [1025], 16, 16, 64, dict(causal=False)),
    ([130], [1500], 1, 1, 128, dict(window=1)),
    ([12, 70], [1300, 70], 20, 1, 64, dict(slack=3)),            # a group of 20: ten heads to a row set
    ([60, 200, 9], [60, 200, 9], 5, 1, 128, dict(slack=4, prefix=[5, 0, 100])),
]


@pytest.mark.parametrize("nq,nk,hq,hk,d,kw", CASES)
def test_prompt_matches_oracle(nq, nk, hq, hk, d, kw):
    run(sum(nq) + sum(nk) + hq + d, nq, nk, hq, hk, d, **kw)


@pytest.mark.parametrize("nq,nk,kw", [
    ([50], [20], dict(causal=False)),
    ([50], [20], dict(prefix=[7])),
    ([300, 4], [40, 900], dict(causal=False, slopes=True)),
    ([9], [1200], dict()),
])
def test_prompt_window_of_any_size(nq, nk, kw):
    """The largest window masks nothing, for queries before the first key (at negative positions) as well."""
    wide, _ = run(31, nq, nk, 4, 2, 64, window=2 ** 31 - 1, **kw)
    none, _ = run(31, nq, nk, 4, 2, 64, **kw)
    assert bool((wide == none).all())


@pytest.mark.parametrize("nq,nk,bad,d,softcap", [(40, 40, 7, 64, 0.0), (300, 300, 0, 128, 5.0), (9, 4000, 8, 128, 0.0), (200, 3000, 150, 64, 0.0)])
def test_prompt_query_with_nan_shows_and_stays_alone(nq, nk, bad, d, softcap):
    """A NaN in a query's row makes that row and its lse NaN, split keys or not; the other rows are bit for bit the same."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(nq + nk)
    q, k, v = dev_bf16(g.standard_normal((nq, 4, d))), dev_bf16(g.standard_normal((nk, 2, d))), dev_bf16(g.standard_normal((nk, 2, d)))
    desc = B.prompt_desc(1, 4, 2, d, nq, nk, nq, nk)
    ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    res = []
    for x in (1.0, float("nan")):
        q[bad, 1, 5] = x
        out, lse = torch.empty_like(q), torch.empty(nq, 4, dtype=torch.float32, device="cuda")
        B.oscar_prompt_attention(desc, q, k, v, i32([0, nq]), i32([0, nk]), out, ws, score=B.score_desc(0.0, softcap, 0, None), lse=lse)
        res.append((out, lse))
    torch.cuda.synchronize()
    (out, lse), (out_n, lse_n) = res
    assert bool(out_n[bad, 1].isnan().all()) and bool(lse_n[bad, 1].isnan())
    out_n[bad, 1], lse_n[bad, 1] = out[bad, 1], lse[bad, 1]
    assert bool((out == out_n).all()) and bool((lse == lse_n).all())


@pytest.mark.parametrize("nq,nk,window,prefix,d,kw", [
    (24, 2000, 300, 0, 128, {}),                       # split keys, alternate tiles
    (24, 2000, 300, 70, 64, {}),
    (200, 700, 150, 65, 64, dict(softcap=4.0)),
    (200, 700, 150, 330, 128, {}),                     # the prefix ends in the window's first tile
    (200, 700, 150, 256, 128, dict(slopes=True)),
    (300, 1500, 40, 0, 128, dict(causal=0)),
    (2, 129, 1, 5, 64, {}),
    (1, 1025, 1, 0, 128, {}),
    (513, 513 + 384, 128, 10, 128, {}),
    (130, 260, 5, 300, 64, {}),                        # the prefix is all keys
])
def test_prompt_rows_before_the_window_may_hold_anything(nq, nk, window, prefix, d, kw):
    """Keys and values that no query sees are NaN or infinite; the result is bit for bit that of zeros there."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(nq + nk + window)
    q, k, v = dev_bf16(g.standard_normal((nq, 4, d))), dev_bf16(g.standard_normal((nk, 2, d))), dev_bf16(g.standard_normal((nk, 2, d)))
    slopes = torch.full((4,), 0.25, device="cuda") if kw.get("slopes") else None
    desc = B.prompt_desc(1, 4, 2, d, nq, nk, nq, nk, bool(kw.get("causal", 1)))
    ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    lo, hi = min(prefix, nk), max(min(prefix, nk), nk - nq - window + 1)
    res = []
    for a, b in ((0.0, 0.0), (float("nan"), float("inf")), (float("-inf"), float("nan"))):
        k[lo:hi], v[lo:hi] = a, b
        out, lse = torch.empty_like(q), torch.empty(nq, 4, dtype=torch.float32, device="cuda")
        B.oscar_prompt_attention(desc, q, k, v, i32([0, nq]), i32([0, nk]), out, ws, prefix_len=i32([prefix]), lse=lse,
                                 score=B.score_desc(0.0, kw.get("softcap", 0.0), window, slopes))
        res.append((out, lse))
    torch.cuda.synchronize()
    assert bool(res[0][0].isfinite().all())
    for out, lse in res[1:]:
        assert bool((out == res[0][0]).all()) and bool((lse == res[0][1]).all())


def test_prompt_clamps_and_reports_bad_rows():
    """Lengths above the bounds and rows outside the tensors are clamped and reported; other requests are not affected."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(4)
    q, k, v = (dev_bf16(g.standard_normal((60, h, 64))) for h in (4, 2, 2))

    def call(cu_q, cu_k, max_q, max_k):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        desc = B.prompt_desc(2, 4, 2, 64, max_q, max_k, 60, 60, True, st)
        w = torch.zeros(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, 9.0)
        B.oscar_prompt_attention(desc, q, k, v, i32(cu_q), i32(cu_k), out, w)
        torch.cuda.synchronize()
        return out, int(st.item())
    good, status = call([0, 20, 50], [0, 20, 50], 30, 30)
    assert status == 0 and bool((good[50:] == 9.0).all())
    for cu_q, cu_k, mq, mk in (([0, 20, 70], [0, 20, 60], 60, 60), ([0, 20, 10], [0, 20, 50], 30, 30), ([0, 20, 50], [0, 20, 50], 20, 30),
                               ([0, 20, 50], [0, 20, 90], 30, 60), ([0, 20, 30], [0, 20, -5], 30, 30)):
        out, status = call(cu_q, cu_k, mq, mk)
        assert status == 2
        assert bool((out[:20] == good[:20]).all())


def test_prompt_on_another_stream_and_in_a_graph():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(6)
    q, k, v = (dev_bf16(g.standard_normal((200, h, 128))) for h in (8, 2, 2))
    desc = B.prompt_desc(1, 8, 2, 128, 200, 200, 200, 200)
    cu = i32([0, 200])
    ws = [torch.zeros(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros_like(q) for _ in range(2)]
    B.oscar_prompt_attention(desc, q, k, v, cu, cu, out[0], ws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        B.oscar_prompt_attention(desc, q, k, v, cu, cu, out[1], ws[1])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert bool((out[0] == out[1]).all())


def test_prompt_scores_far_apart_and_rows_of_one_key():
    """Scores of thousands (one key takes all), a whole row of equal scores, and caps that bite."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(8)
    n, hq, hk, d = 300, 4, 2, 64
    q, k, v = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    q[:100] *= 512.0
    q[100:150] = 0.0
    for softcap in (0.0, 2.0, 4000.0):
        desc = B.prompt_desc(1, hq, hk, d, n, n, n, n)
        ws = torch.zeros(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        B.oscar_prompt_attention(desc, dev_bf16(q), dev_bf16(k), dev_bf16(v), i32([0, n]), i32([0, n]), out, ws,
                                 score=B.score_desc(softcap=softcap))
        got = host(out)
        for h in range(hq):
            r, r_abs, _ = O.masked_attention(O.modified_scores(q[:, h], k[:, h // 2], 0, softcap=softcap), v[:, h // 2])
            # fp32 scores of up to 2^13 are off by up to 2^-10 each, which their weights repeat
            assert (np.abs(got[:, h] - r) <= HALF_BF16 * (np.abs(r) + r_abs) + 2.0 ** -9 * r_abs + 2.0 ** -14).all()


def spoil(d, size):
    """Leaves queries of the given size in every SM's shared memory: all rows of every tile, whatever its head group."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(1)
    b, n = 400, 64
    q = (torch.randn(b * n, 4, d, generator=g, device="cuda") * size).to(torch.bfloat16)
    k = torch.randn(b * n, 1, d, generator=g, device="cuda").to(torch.bfloat16)
    desc = B.prompt_desc(b, 4, 1, d, n, n, b * n, b * n)
    ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    cu = i32(np.arange(b + 1) * n)
    B.oscar_prompt_attention(desc, q, k, k, cu, cu, torch.empty_like(q), ws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 40.0])
@pytest.mark.parametrize("group,nq,nk", [(3, 200, 700), (5, 300, 1000), (6, 31, 600), (7, 9, 4000), (15, 3, 5000)])
def test_prompt_bits_do_not_depend_on_the_calls_before(group, nq, nk, softcap, d):
    """A group that does not divide 128 leaves rows of a query tile over: what an earlier call left there has no say."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(group + nk)
    q, k, v = (dev_bf16(g.standard_normal((n, h, d))) for n, h in ((nq, group), (nk, 1), (nk, 1)))
    desc = B.prompt_desc(1, group, 1, d, nq, nk, nq, nk)
    ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    res = []
    for size in (0.0, 300.0, 1.0, 1e6):
        spoil(d, size)
        out, lse = torch.empty_like(q), torch.empty(nq, group, dtype=torch.float32, device="cuda")
        B.oscar_prompt_attention(desc, q, k, v, i32([0, nq]), i32([0, nk]), out, ws, score=B.score_desc(softcap=softcap), lse=lse)
        torch.cuda.synchronize()
        res.append((out, lse))
    for out, lse in res[1:]:
        assert bool((out == res[0][0]).all()) and bool((lse == res[0][1]).all())


@pytest.mark.parametrize("hq,softcap", [(4, 0.0), (4, 40.0), (3, 40.0), (8, 0.0)])
def test_prompt_rows_do_not_reach_one_another(hq, softcap):
    """Another request's queries and keys, or another query row of one's own, change no bit of a row, whatever their size."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g, d = np.random.default_rng(hq), 64
    nq, nk = [40, 50], [700, 300]
    q, k, v = (dev_bf16(g.standard_normal((n, h, d))) for n, h in ((90, hq), (1000, 1), (1000, 1)))
    desc = B.prompt_desc(2, hq, 1, d, 50, 700, 90, 1000)
    ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    res = []
    for size in (1.0, 300.0, 2.0 ** -20):
        a, b = q.clone(), k.clone()
        a[40:] *= size
        a[7, 0] *= size
        b[700:] *= size
        out, lse = torch.empty_like(q), torch.empty(90, hq, dtype=torch.float32, device="cuda")
        B.oscar_prompt_attention(desc, a, b, v, i32([0, 40, 90]), i32([0, 700, 1000]), out, ws, score=B.score_desc(softcap=softcap),
                                 lse=lse)
        out[7, 0], lse[7, 0] = 0.0, 0.0
        res.append((out[:40], lse[:40]))
    torch.cuda.synchronize()
    for out, lse in res[1:]:
        assert bool((out == res[0][0]).all()) and bool((lse == res[0][1]).all())


@pytest.mark.parametrize("softcap", [1e3, 1e5, 1e7, 1e12, 1e30, 1e38])
def test_prompt_large_caps_leave_ordinary_scores(softcap):
    """Scores of ordinary size under a cap far above them, with and without a row at the cap in the same warp: the
    tolerances are those of the other cases."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g, n, hq, d = np.random.default_rng(12), 200, 4, 64
    q, k, v = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, 1, 1))
    for far in (False, True):
        if far:
            q[::9] *= 2.0 ** np.ceil(np.log2(min(softcap, 1e6)))
        desc = B.prompt_desc(1, hq, 1, d, n, n, n, n)
        ws = torch.empty(B.oscar_prompt_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        B.oscar_prompt_attention(desc, dev_bf16(q), dev_bf16(k), dev_bf16(v), i32([0, n]), i32([0, n]), out, ws,
                                 score=B.score_desc(softcap=softcap))
        got = host(out)
        rows = np.arange(n) % 9 != 0 if far else np.ones(n, bool)
        for h in range(hq):
            r, r_abs, _ = O.masked_attention(O.modified_scores(q[:, h], k[:, 0], 0, softcap=softcap), v[:, 0])
            assert (np.abs(got[:, h] - r) <= HALF_BF16 * (np.abs(r) + r_abs) + 2.0 ** -14)[rows].all()
