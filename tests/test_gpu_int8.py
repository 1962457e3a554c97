"""8-bit layers and rotary positions on the GPU against the float64 oracle: angle
tables, norm and rotation, append, read back, decode attention, and a run of them
together.

Tolerances.  Codes, scales, zeros and held rows are compared exactly with the
oracle's of the rotated row that the kernel itself returned.
 - A table entry: polynomials to 2e-9, an argument and a value of 24 bits with a handful
   of fp32 operations: 2^-21 of the entry's size (a sine near 0 keeps its bits: its argument
   has 24 at any size), and 2^-30 of 2 pi for what doubles in the oracle's own quarter lose.
 - A rotated row: one bf16 rounding (2^-8) of an fp32 sum of two products; each has about six
   roundings (weight by angle, channel, the sum of squares of 128, a root to 2 ulp, the
   product with it): 2^-19 of the terms' sizes covers them.
 - The decode's output: one bf16 rounding (2^-8).  A score is an fp32 sum of at most 128
   products, off by 2^-22 of scale sum |q| (255 s + 2 |z|) < 128 here, so 2^-15 of each weight,
   with its power (2^-22), 22 bits of the product with the value's scale, and at most
   600 additions of fp32 (2^-23 each in the tensor cores): 2^-15 + 600 2^-23 < 2^-13
   of (softmax weight) (|value| + |zero|) <= 2^-12 max |value|.  The logarithm of the sum: 2^-13.
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


def dev_f32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def host(t):
    return t.double().cpu().numpy()


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def angles(n, rot, theta=1e4):
    f = theta ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Layer:
    """An 8-bit layer of requests of the given lengths, its pages shuffled and every unused slot stale (NaN pairs)."""

    def __init__(self, seed, lens, hq, hk, d, fill=True, extra_pages=2, max_pages=None, tau=65504.0, shift=0.3):
        import torch
        from bit_rotated_kv_split_gb300.cache import Int8Cache
        self.g = np.random.default_rng(seed)
        self.lens, self.hq, self.hk, self.d = list(lens), hq, hk, d
        pages = [-(-n // 16) for n in lens]
        n_pages = sum(pages) + extra_pages
        self.cache = Int8Cache(len(lens), hq, hk, d, max_pages or max(max(pages), 1), n_pages, tau_k=tau, tau_v=tau)
        order = self.g.permutation(n_pages)
        self.table = np.full((len(lens), self.cache.max_pages_per_seq), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.pool = np.full((n_pages, hk, O.int8_block_bytes(d)), 0xFF, np.uint8)
        self.k, self.v = [], []
        if fill:
            for b, n in enumerate(lens):
                k = O.bf16(self.g.standard_normal((n, hk, d)) * np.where(self.g.random((1, hk, d)) < 0.05, 4, 1))
                v = O.bf16(self.g.standard_normal((n, hk, d)) + shift)
                self.k.append(self.put(b, np.arange(n), 0, k)), self.v.append(self.put(b, np.arange(n), 1, v))
        self.cache.page_table.copy_(torch.from_numpy(self.table))
        self.cache.seq_len.copy_(i32(lens))
        self.upload()
        self.desc = self.cache.desc(max(max(lens), 0))

    def upload(self):
        import torch
        self.cache.pages.copy_(torch.from_numpy(self.pool.reshape(-1)))

    def put(self, b, pos, which, rows):
        """Quantises and stores rows [n][hk][d] at positions pos; returns what they stand for."""
        c, s, z = O.int8_quantize(rows, self.cache.tau_k)
        pos = np.asarray(pos, dtype=np.int64)
        O.int8_store_rows(self.pool, self.table[b, pos // 16], pos % 16, which, c, s, z)
        return O.int8_values(c, s, z)

    def gpu_pool(self):
        return self.cache.pages.cpu().numpy().reshape(self.pool.shape)

    def status(self):
        return int(self.cache.dev_status.item())


# ---------------------------------------------------------------- angle tables

@pytest.mark.parametrize("rot,n,first", [(16, 1, 0), (64, 4099, 0), (96, 77, 12345), (128, 300, 2 ** 20 - 7), (32, 33, 2 ** 31 + 5),
                                         (128, 9, 2 ** 39 + 3), (48, 40000, 5)])
@pytest.mark.parametrize("magnitude", [1.0, 1.1386294361119891])
def test_table_matches_oracle(rot, n, first, magnitude):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    freq, _ = B.oscar_rope_frequencies(rot, 1e6, "by_index", 4.0, 32768.0)
    freq[1] = 6.0                                    # an arbitrary one, most of a turn a position
    out = torch.full((n + 1, rot), -9.0, dtype=torch.float32, device="cuda")
    B.oscar_rope_table(freq, out[:n], magnitude=magnitude, first=first)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.arange(min(n, 70)), np.random.default_rng(n).integers(0, n, 40), [n - 1]]))
    want = np.concatenate([O.rope_table(freq, first + int(j), 1, magnitude) for j in rows])
    got = host(out)[rows]
    # (a position's turns carry (first + j) 2^-64)
    near = 2.0 ** -21 * np.abs(want) + 2.0 ** -50 + 2 * np.pi * (first + n) * 2.0 ** -64 * magnitude
    assert (np.abs(got - want) <= near).all()
    assert (out[n] == -9.0).all()


@pytest.mark.parametrize("magnitude", [1.0, -3.0])
def test_table_far_positions_within_half_a_step_a_position(magnitude):
    """Sines next to 0 near 2^40 positions: what the step's rounding to 2^-64 of a turn leaves, (first + j) 2^-65, shows there."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    freq, _ = B.oscar_rope_frequencies(128, 1e6)
    two_pi = 6283185307179586476925286766559005768394338798750211641949889   # times 10^-60
    turns = []                                       # of one position, times 2^200
    for w in freq:
        num, den = float(w).as_integer_ratio()
        turns.append(num * 10 ** 60 * 2 ** 200 // (den * two_pi))
    seen = 0
    for i, t in enumerate(turns):
        at = range(2 ** 40 - 20000, 2 ** 40)
        first = min(at, key=lambda p: min(p * t % 2 ** 200, -p * t % 2 ** 200))
        out = torch.empty(1, 128, dtype=torch.float32, device="cuda")
        B.oscar_rope_table(freq, out, magnitude=magnitude, first=first)
        want = O.rope_table(freq, first, 1, magnitude)
        near = 2.0 ** -21 * np.abs(want) + (2 * np.pi * first * 2.0 ** -65 + 2.0 ** -50) * abs(magnitude)
        assert (np.abs(host(out) - want) <= near).all(), i
        # the test sees a step off by more than that: the sine's own part of the bound is far below
        seen += 2.0 ** -21 * abs(want[0, 64 + i]) < 0.2 * 2 * np.pi * first * 2.0 ** -66 * abs(magnitude)
    assert seen > 20


# ---------------------------------------------------------------- norm and rotation

def rotated(x, weight, cs, inter, eps=1e-6):
    """(the row in float64, the sizes of its terms)."""
    y = O.head_norm(x, weight, eps)
    t = np.abs(y)
    rot = cs.shape[1]
    if rot:
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        t = t.copy()
        t[..., a] = t[..., b] = t[..., a] + t[..., b]
    return O.rope(y, cs, inter), t * max(1.0, np.abs(cs).max() if rot else 1.0)


ROWS = [
    # d, hq, hk, rot, interleaved, n, weights, mode
    (128, 32, 8, 128, False, 1, "qk", "packed"),
    (128, 8, 2, 128, True, 21, "qk", "apart"),
    (128, 5, 5, 32, False, 33, "", "packed"),
    (64, 4, 4, 64, False, 23, "q", "in place"),
    (64, 9, 3, 16, True, 41, "k", "apart"),
    (64, 1, 1, 0, False, 2, "qk", "apart"),
    (128, 48, 3, 64, False, 181, "qk", "in place"),
    (128, 7, 1, 96, True, 700, "qk", "packed"),
    (64, 16, 8, 48, False, 1300, "", "apart"),
]


@pytest.mark.parametrize("d,hq,hk,rot,inter,n,weights,mode", ROWS)
def test_norm_rope_matches_oracle(d, hq, hk, rot, inter, n, weights, mode):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    g = np.random.default_rng(d + hq + n)
    q, k = (O.bf16(g.standard_normal((n, h, d)) * s) for h, s in ((hq, 1.0), (hk, 3.0)))
    q[0, 0] = 0.0
    wq, wk = (O.bf16(1 + 0.3 * g.standard_normal(d)) if c in weights else None for c in "qk")
    norm = B.norm_desc(*(None if w is None else dev_bf16(w) for w in (wq, wk)), eps=1e-5) if weights else None
    cs = angles(500, rot)
    rope = B.rope_desc(dev_f32(cs), rot, inter) if rot else None
    pos = g.integers(0, 500, n)
    qkv = dev_bf16(np.concatenate([q, k, k[:, :1]], 1))
    tq, tk, _ = qkv.split([hq, hk, 1], 1)
    if mode == "apart":
        tq, tk = dev_bf16(q), dev_bf16(k)
    q_out, k_out = (tq, tk) if mode == "in place" else (torch.full((n, h, d), -7.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.oscar_norm_rope(norm, rope, tq, tk, i32(pos) if rot else None, q_out, k_out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for got, x, w in ((q_out, q, wq), (k_out, k, wk)):
        want, terms = rotated(x, w, cs[pos], inter, 1e-5)
        assert (np.abs(host(got) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms + 1e-38).all()
    assert torch.equal(qkv[:, -1].float().cpu(), torch.from_numpy(k[:, 0]).float())    # its neighbours are as they were
    if mode == "apart":
        one = torch.empty_like(k_out)
        B.oscar_norm_rope(norm, rope, None, tk, i32(pos) if rot else None, None, one)
        two = torch.empty_like(q_out)
        B.oscar_norm_rope(norm, rope, tq, None, i32(pos) if rot else None, two, None)
        assert torch.equal(one, k_out) and torch.equal(two, q_out)


def test_norm_rope_skips_and_flags():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, d = 6, 64
    rope = B.rope_desc(dev_f32(angles(10, d)), d)
    q, k = (dev_bf16(np.random.default_rng(h).standard_normal((n, h, d))) for h in (4, 2))
    pos = i32([3, -1, 9, 10, -2, 0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = torch.full_like(q, -7.0), torch.full_like(k, -7.0)
    B.oscar_norm_rope(None, rope, q, k, pos, qo, ko, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.DEV_LENGTH
    for i in (1, 3, 4):
        assert (qo[i] == -7.0).all() and (ko[i] == -7.0).all()
    for i in (0, 2, 5):
        assert not (qo[i] == -7.0).any()
    status.zero_()
    B.oscar_norm_rope(None, rope, q, k, i32([3, -1, 9, 1, -1, 0]), qo, ko, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0                   # a padding row is no fault
    B.oscar_norm_rope(None, rope, q, k, pos, qo, ko)   # and without the word
    torch.cuda.synchronize()
    # without a rotation a position says only whether the row is padding
    qo.fill_(-7.0), ko.fill_(-7.0)
    w = dev_bf16(np.ones(d))
    B.oscar_norm_rope(B.norm_desc(w, w), None, q, k, i32([3, -1, 9, 10 ** 9, -2, 0]), qo, ko, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (qo[1] == -7.0).all() and (ko[1] == -7.0).all()
    assert not (qo[[0, 2, 3, 4, 5]] == -7.0).any()


def test_norm_rope_bad_values_stay_in_their_rows():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    n, d = 3, 128
    g = np.random.default_rng(5)
    x = dev_bf16(g.standard_normal((n, 4, d)))
    w = dev_bf16(np.ones(d))
    rope = B.rope_desc(dev_f32(angles(8, 64)), 64)
    good, bad = torch.empty_like(x), torch.empty_like(x)
    B.oscar_norm_rope(None, rope, x, None, i32([1, 2, 3]), good, None)
    y = x.clone()
    y[1, 2, 100] = float("inf")                      # of a channel that does not turn
    y[2, 1, 3] = float("nan")
    B.oscar_norm_rope(None, rope, y, None, i32([1, 2, 3]), bad, None)
    torch.cuda.synchronize()
    same = (good == bad)
    assert same[0].all() and same[1, [0, 1, 3]].all() and same[2, [0, 2, 3]].all()
    assert bad[1, 2, 100] == float("inf") and same[1, 2, :100].all() and same[1, 2, 101:].all()
    assert (~same[2, 1]).nonzero().flatten().tolist() == [3, 35] and bad[2, 1, [3, 35]].isnan().all()
    B.oscar_norm_rope(B.norm_desc(w), rope, y, None, i32([1, 2, 3]), bad, None)
    torch.cuda.synchronize()
    assert bad[2, 1].isnan().all() and not bad[2, [0, 2, 3]].isnan().any() and not bad[0].isnan().any()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 1e-20])
def test_norm_of_the_smallest_rows(eps, inter):
    """Rows of every size down to bf16's least number, whose squares are below fp32: normed as larger ones are; rows of zeros
    stay zeros, with no eps either."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, hq, hk = 128, 5, 2
    g = np.random.default_rng(6)
    sizes = [-133, -132, -128, -126, -120, -100, -80, -75, -70, -64, -60, -50, -46, -45, -44, -43, -40, -30, 0]
    n = len(sizes) + 1
    q, k = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, hk))
    for x in (q, k):
        for i, e in enumerate(sizes):
            y = x[i] * 2.0 ** e                      # (below 2^-126 bf16 keeps multiples of 2^-133)
            x[i] = np.where(np.abs(y) < 2.0 ** -126, np.rint(y * 2.0 ** 133) * 2.0 ** -133, y)
        x[-1] = 0.0
        x[3, 0] = 0.0
        x[3, 0, 77] = 2.0 ** -133                    # one channel alone, the least there is
        x[4, 1] = 2.0 ** -80                         # a constant row
    eps = float(np.float32(eps))
    wq, wk = (O.bf16(1 + 0.3 * g.standard_normal(d)) for _ in range(2))
    norm = B.norm_desc(dev_bf16(wq), dev_bf16(wk), eps)
    cs = angles(50, 64)
    pos = g.integers(0, 50, n)
    tq, tk = dev_bf16(q), dev_bf16(k)
    assert (host(tq) == q).all() and (host(tk) == k).all()
    qo, ko = torch.empty_like(tq), torch.empty_like(tk)
    B.oscar_norm_rope(norm, B.rope_desc(dev_f32(cs), 64, inter), tq, tk, i32(pos), qo, ko)
    torch.cuda.synchronize()
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        zeros = (x == 0).all(-1, keepdims=True)
        want, terms = rotated(np.where(zeros, 1.0, x), w, cs[pos], inter, eps)
        want, terms = np.where(zeros, 0.0, want), np.where(zeros, 0.0, terms)
        # below bf16's normal range a result is off by half a step of 2^-133; where eps makes them small, two products
        # of a row's numbers below fp32's normal range by half of 2^-149 each, times the root
        near = 2.0 ** -134 + (2.0 ** -149 / np.sqrt(eps) if eps > 2.0 ** -90 else 0.0) * np.abs(w).max()
        assert (np.abs(host(got) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms + near).all()


# ---------------------------------------------------------------- append and read back

APPENDS = [
    # d, hq, hk, rot, interleaved, tokens of each request, tau, norm
    (128, 32, 8, 128, False, [1], 65504.0, True),
    (128, 8, 2, 128, True, [3, 1, 17], 65504.0, False),
    (128, 5, 5, 32, False, [33], 2.0, True),
    (64, 4, 4, 64, False, [7, 16], 65504.0, True),
    (64, 9, 3, 16, True, [40, 1], 65504.0, True),
    (64, 1, 1, 0, False, [2], 65504.0, False),
    (128, 48, 3, 64, False, [150, 31], 65504.0, True),
    (64, 24, 8, 64, False, [900, 1, 333], 65504.0, False),
]


@pytest.mark.parametrize("d,hq,hk,rot,inter,tokens,tau,normed", APPENDS)
@pytest.mark.parametrize("packed", [True, False])
def test_append_matches_oracle(d, hq, hk, rot, inter, tokens, tau, normed, packed):
    """The new tokens' pages, held rows, k' and q'; every other byte of the pool as it was; and the rows read back."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    past = [5 * (i + 1) for i in range(len(tokens))]
    L = Layer(d + hq, [p + t for p, t in zip(past, tokens)], hq, hk, d, fill=False, tau=tau)
    n, g = sum(tokens), L.g
    req = np.repeat(np.arange(len(tokens)), tokens)
    pos = np.concatenate([np.arange(p, p + t) for p, t in zip(past, tokens)])
    perm = g.permutation(n)
    req, pos = req[perm], pos[perm]
    q, k, v = (O.bf16(g.standard_normal((n, h, d)) * s) for h, s in ((hq, 1.0), (hk, 3.0), (hk, 1.0)))
    v[0, 0] = 0.0                                   # constant rows: that fp16 holds, and not
    if n > 3:
        v[1, 0], v[2, 0], v[3, 0] = 1.5, O.bf16(1e-9), O.bf16(-3e-9)
        v[1, -1] = O.bf16(2.0 ** -22 * g.standard_normal(d))      # subnormal scales
        v[2, -1, 0] = 60000.0                                     # one far channel
        v[3, -1] += 512.0                                         # a range far from 0
    v = O.bf16(v)                                   # (as the rows are handed over)
    wq, wk = (O.bf16(1 + 0.3 * g.standard_normal(d)) if normed else None for _ in range(2))
    norm = B.norm_desc(dev_bf16(wq), dev_bf16(wk)) if normed else None
    tq, tk, tv = dev_bf16(np.concatenate([q, k, v], 1)).split([hq, hk, hk], 1) if packed else (dev_bf16(q), dev_bf16(k), dev_bf16(v))
    cs = angles(int(pos.max()) + 300, rot)
    rope_pos = pos + g.integers(0, 300, n) if not packed else pos
    rope = B.rope_desc(dev_f32(cs), rot, inter)
    out = {x: torch.full((n, h, d), -7.0, dtype=torch.bfloat16, device="cuda") for x, h in (("q_out", hq), ("k_out", hk), ("k_held", hk), ("v_held", hk))}
    B.oscar_rope_append_int8(L.desc, norm, rope, tq, tk, tv, i32(req), i32(pos), rope_pos=None if packed else i32(rope_pos), **out)
    torch.cuda.synchronize()
    assert L.status() == 0
    for name, x, w in (("q_out", q, wq), ("k_out", k, wk)):
        want, terms = rotated(x, w, cs[rope_pos], inter)
        assert (np.abs(host(out[name]) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms).all(), name
    held = []
    for which, rows in ((0, host(out["k_out"])), (1, v)):
        c, s, z = O.int8_quantize(rows, tau)
        O.int8_store_rows(L.pool, L.table[req, pos // 16], pos % 16, which, c, s, z)
        held.append(O.bf16(O.int8_values(c, s, z)))
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)
    np.testing.assert_array_equal(host(out["k_held"]), held[0])
    np.testing.assert_array_equal(host(out["v_held"]), held[1])
    # read back, strided rows
    both = torch.full((n, 2 * hk, d), -7.0, dtype=torch.bfloat16, device="cuda")
    B.oscar_gather_int8(L.desc, i32(req), i32(pos), both[:, :hk], both[:, hk:])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(both), np.concatenate(held, 1))


def test_append_in_place_and_alone():
    """q and k written over, held rows over v; and neither q nor any output."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, hq, hk, n = 128, 8, 4, 37
    L, M = (Layer(3, [n], hq, hk, d, fill=False) for _ in range(2))
    g = np.random.default_rng(1)
    q, k, v = (dev_bf16(g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    w = dev_bf16(1 + 0.1 * g.standard_normal(d))
    norm, rope = B.norm_desc(w, w), B.rope_desc(dev_f32(angles(n, d)), d)
    req, pos = i32(np.zeros(n)), i32(np.arange(n))
    want = [torch.empty_like(x) for x in (q, k, k, v)]
    B.oscar_rope_append_int8(L.desc, norm, rope, q, k, v, req, pos, want[0], want[1], k_held=want[2], v_held=want[3])
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    B.oscar_rope_append_int8(M.desc, norm, rope, q2, k2, v2, req, pos, q2, k2, v_held=v2)
    torch.cuda.synchronize()
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1]) and torch.equal(v2, want[3])
    np.testing.assert_array_equal(L.gpu_pool(), M.gpu_pool())
    k3 = k.clone()
    M.upload()
    B.oscar_rope_append_int8(M.desc, norm, rope, None, k3, v, req, pos, None, k_held=k3)
    torch.cuda.synchronize()
    assert torch.equal(k3, want[2])
    np.testing.assert_array_equal(L.gpu_pool(), M.gpu_pool())
    B.oscar_rope_append_int8(M.desc, None, None, None, k, v, req, pos, None)
    torch.cuda.synchronize()
    c, s, z = O.int8_quantize(host(k))
    O.int8_store_rows(L.pool, L.table[0, np.arange(n) // 16], np.arange(n) % 16, 0, c, s, z)
    at = O.int8_code_byte(d, 0, 3, np.arange(d))
    np.testing.assert_array_equal(M.gpu_pool()[L.table[0, 0]][:, at], L.pool[L.table[0, 0]][:, at])


def test_codes_at_ties_and_borders():
    """Quotients at, and just beside, halves; ranges whose scale lies at a border of fp16."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, n = 64, 512
    g = np.random.default_rng(11)
    # integers of at most 8 bits over a power of two, with 0 and 255 / 2 present: scale 1/2 or so, codes and halves exact
    x = g.integers(0, 256, (n, 1, d)) / 2.0
    x[:, :, 0], x[:, :, 1] = 0.0, 127.5
    x[n // 2:] *= 2.0 ** g.integers(-20, 8, (n // 2, 1, 1))
    y = O.bf16(g.integers(-255, 256, (n, 1, d)) * 2.0 ** g.integers(-14, 6, (n, 1, 1)))
    y[::3] = O.bf16(y[::3] * 3.7)
    y[1::3, :, 5] = O.bf16(2.0 ** 15 * g.standard_normal((len(y[1::3]), 1)))
    L = Layer(2, [n], 1, 1, d, fill=False)
    B.oscar_rope_append_int8(L.desc, None, None, None, dev_bf16(O.bf16(x)), dev_bf16(y), i32(np.zeros(n)), i32(np.arange(n)), None)
    torch.cuda.synchronize()
    for which, rows in ((0, O.bf16(x)), (1, y)):
        c, s, z = O.int8_quantize(rows)
        O.int8_store_rows(L.pool, L.table[0, np.arange(n) // 16], np.arange(n) % 16, which, c, s, z)
        assert (np.abs(O.int8_values(c, s, z) - np.clip(rows, -65504.0, 65504.0)) <= s.astype(float)[..., None] / 2).all()
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


def test_append_skips_and_flags():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, hq, hk = 64, 2, 2
    L = Layer(9, [40, 20], hq, hk, d, fill=False, max_pages=4)
    rope = B.rope_desc(dev_f32(angles(30, d)), d)
    g = np.random.default_rng(2)
    cases = [  # request, position, rotation row, page id planted, bit
        (-1, 3, 3, None, 0), (2, 3, 3, None, B.DEV_LENGTH), (-2, 3, 3, None, B.DEV_LENGTH), (0, 64, 3, None, B.DEV_LENGTH),
        (0, -1, 3, None, B.DEV_LENGTH), (0, 3, 30, None, B.DEV_LENGTH), (0, 3, -1, None, B.DEV_LENGTH),
        (1, 40, 3, None, B.DEV_PAGE_BOUNDS), (1, 3, 3, 1000, B.DEV_PAGE_BOUNDS), (-1, -5, 99, None, 0),
    ]
    for req, pos, row, page, bit in cases:
        table = L.table.copy()
        if page is not None:
            table[1, 0] = page
        L.cache.page_table.copy_(torch.from_numpy(table))
        L.cache.dev_status.zero_()
        q, k, v = (dev_bf16(g.standard_normal((1, h, d))) for h in (hq, hk, hk))
        out = [torch.full_like(x, -7.0) for x in (q, k, k, v)]
        B.oscar_rope_append_int8(L.desc, None, rope, q, k, v, i32([req]), i32([pos]), out[0], out[1], rope_pos=i32([row]),
                                 k_held=out[2], v_held=out[3])
        if row == 3:
            got = [torch.full_like(k, -7.0) for _ in range(2)]
            B.oscar_gather_int8(L.desc, i32([req]), i32([pos]), *got)
            out += got
        torch.cuda.synchronize()
        assert L.status() == bit, (req, pos, row)
        assert all((x == -7.0).all() for x in out)
        np.testing.assert_array_equal(L.gpu_pool(), L.pool)


def test_append_nan_and_infinity_stay_in_their_rows():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, hk, n = 128, 2, 4
    L = Layer(1, [n], 2, hk, d, fill=False, tau=100.0)
    g = np.random.default_rng(4)
    k, v = (O.bf16(g.standard_normal((n, hk, d))) for _ in range(2))
    tk, tv = dev_bf16(k), dev_bf16(v)
    tk[1, 0, 7], tv[2, 1, 3], tv[3, 0, 0] = float("nan"), float("-inf"), float("inf")
    k[1, 0, 7], v[2, 1, 3], v[3, 0, 0] = -100.0, -100.0, 100.0
    B.oscar_rope_append_int8(L.desc, None, None, None, tk, tv, i32(np.zeros(n)), i32(np.arange(n)), None)
    torch.cuda.synchronize()
    for which, rows in ((0, k), (1, v)):
        O.int8_store_rows(L.pool, L.table[0, [0] * n], np.arange(n), which, *O.int8_quantize(rows, 100.0))
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


def test_append_of_a_key_of_zeros_without_eps():
    """Its page holds zeros (a NaN would stand there as -tau)."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, hk, n = 64, 3, 5
    L = Layer(17, [n], hk, hk, d, fill=False)
    k, v = (O.bf16(L.g.standard_normal((n, hk, d))) for _ in range(2))
    k[2, 1], k[3] = 0.0, 0.0
    k[4, 2] = 2.0 ** -90
    w = dev_bf16(np.ones(d))
    k_out = torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda")
    B.oscar_rope_append_int8(L.desc, B.norm_desc(w, w, 0.0), None, None, dev_bf16(k), dev_bf16(v), i32(np.zeros(n)), i32(np.arange(n)), None, k_out)
    torch.cuda.synchronize()
    assert (k_out[2, 1] == 0).all() and (k_out[3] == 0).all() and (k_out[4, 2] == 1).all()
    L.put(0, np.arange(n), 0, host(k_out)), L.put(0, np.arange(n), 1, v)
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)


# ---------------------------------------------------------------- decode

def decode(L, q, score=None, lse=True, ws=None):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    tq = q if isinstance(q, torch.Tensor) else dev_bf16(q)
    out = torch.full(tq.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(tq.shape[:2], -7.0, dtype=torch.float32, device="cuda") if lse else None
    if ws is None:
        ws = torch.zeros(B.oscar_decode_int8_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda")
    B.oscar_decode_attention_int8(L.desc, tq, out, ws, score=score, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def check_decode(L, q, out, lse, requests=None, **form):
    slopes = form.pop("slopes", None)
    got, got_lse = host(out), host(lse)
    group = L.hq // L.hk
    for b in range(len(L.lens)) if requests is None else requests:
        n = L.lens[b]
        for h in range(L.hq):
            k, v = L.k[b][:, h // group], L.v[b][:, h // group]
            t = O.modified_scores(q[b, h:h + 1], k, n - 1, slope=0.0 if slopes is None else float(slopes[h]), **form)
            want, _, want_lse = O.masked_attention(t, v)
            if n == 0:
                assert (got[b, h] == 0).all() and got_lse[b, h] == -np.inf
                continue
            near = HALF_BF16 * np.abs(want[0]) + 2.0 ** -12 * np.abs(v).max()
            assert (np.abs(got[b, h] - want[0]) <= near).all(), (b, h, n, np.abs(got[b, h] - want[0]).max())
            assert abs(got_lse[b, h] - want_lse[0]) <= 2.0 ** -13 + 2.0 ** -22 * abs(want_lse[0]), (b, h, n)


DECODES = [
    # d, hq, hk, lengths, form
    (128, 4, 1, [1], {}),
    (128, 8, 8, [1, 2, 15, 16, 17, 31, 32, 33, 0, 191, 192, 193], {}),
    (64, 5, 1, [777, 0, 3], {}),
    (64, 16, 1, [100, 1500], {}),
    (128, 32, 2, [333, 48, 784, 5], {}),
    (128, 18, 2, [64, 1025], dict(softcap=5.0)),
    (64, 12, 4, [640, 2, 1111], dict(softcap=30.0, window=100)),
    (128, 16, 2, [500, 1300, 90], dict(window=257)),
    (128, 8, 2, [500, 17, 90], dict(window=1)),
    (64, 40, 8, [301, 1999], dict(window=600, slopes=True)),
    (128, 24, 2, [513, 4], dict(slopes=True, softcap=20.0)),
    (128, 6, 2, [9001, 40], dict(scale=0.2)),
    (64, 9, 3, [6000, 6000, 1], {}),
]


@pytest.mark.parametrize("d,hq,hk,lens,form", DECODES)
def test_decode_matches_oracle(d, hq, hk, lens, form):
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(d + hq + sum(lens), lens, hq, hk, d)
    q = O.bf16(L.g.standard_normal((len(lens), hq, d)))
    form = dict(form)
    if form.get("slopes"):
        form["slopes"] = 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)
        form["slopes"] = form["slopes"].astype(np.float32).astype(np.float64)
    score = B.score_desc(form.get("scale", 0.0), form.get("softcap", 0.0), form.get("window", 0),
                         dev_f32(form["slopes"]) if "slopes" in form else None)
    out, lse = decode(L, q, score)
    assert L.status() == 0
    if "scale" in form:
        form["scale"] = float(np.float32(form["scale"]))
    check_decode(L, q, out, lse, **form)
    again, lse2 = decode(L, q, score)
    assert (again == out).all() and (lse2 == lse).all()         # not by scheduling
    alone, _ = decode(L, q, score, lse=False)
    assert (alone == out).all()


@pytest.mark.parametrize("d,hq,lens", [(128, 4, [2000]), (64, 8, [2999, 100]), (128, 16, [5000, 1, 700])])
def test_decode_loses_no_page(d, hq, lens):
    """Equal weights, and values that mark their page's channel: a page left out or counted twice shows in it."""
    L = Layer(7, lens, hq, 1, d, fill=False)
    for b, n in enumerate(lens):
        v = np.zeros((n, 1, d))
        v[np.arange(n), 0, np.arange(n) // 16 % d] = 1.0
        L.k.append(L.put(b, np.arange(n), 0, O.bf16(L.g.standard_normal((n, 1, d)))))
        L.v.append(L.put(b, np.arange(n), 1, v))
    L.upload()
    out, lse = decode(L, np.zeros((len(lens), hq, d)))
    for b, n in enumerate(lens):
        want = L.v[b][:, 0].mean(0)
        # one page of ceil(n / 16 / d) in its channel: far above the rounding's 2^-8
        assert (np.abs(host(out)[b] - want) <= HALF_BF16 * want + 2.0 ** -20).all()
        np.testing.assert_allclose(host(lse)[b], np.log(n), rtol=2.0 ** -21)


def test_decode_workspace_serves_calls_of_all_sizes():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    small, big = Layer(1, [40, 900], 8, 2, 128), Layer(2, [5000, 3, 2500], 32, 2, 128)
    ws = torch.zeros(B.oscar_decode_int8_workspace_bytes(big.desc), dtype=torch.uint8, device="cuda")
    assert ws.numel() == B.oscar_decode_int8_workspace_bytes(small.desc)
    qs = [O.bf16(L.g.standard_normal((len(L.lens), L.hq, L.d))) for L in (small, big)]
    for L, q in ((small, qs[0]), (big, qs[1]), (small, qs[0])):
        check_decode(L, q, *decode(L, q, ws=ws))


def test_decode_ragged_batch_of_many_short_requests():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 70, 700)]
    L = Layer(5, lens, 4, 2, 64)
    q = O.bf16(L.g.standard_normal((700, 4, 64)))
    out, lse = decode(L, q)
    check_decode(L, q, out, lse)


def test_decode_shared_and_permuted_pages():
    """Two requests on the same pages give the same bits as each alone on copies elsewhere."""
    import torch
    L = Layer(6, [800, 800], 8, 2, 128)
    q = O.bf16(np.repeat(L.g.standard_normal((1, 8, 128)), 2, 0))
    L.table[1] = L.table[0]
    L.cache.page_table.copy_(torch.from_numpy(L.table))
    L.k[1], L.v[1] = L.k[0], L.v[0]
    out, lse = decode(L, q)
    check_decode(L, q, out, lse)


def test_decode_bits_do_not_depend_on_the_places_of_pages():
    """The same blocks at other places of the pool, behind another table: the same bits."""
    import torch
    L = Layer(6, [800, 3000, 17], 8, 2, 128)
    q = O.bf16(L.g.standard_normal((3, 8, 128)))
    out, lse = decode(L, q)
    check_decode(L, q, out, lse)
    for seed in (0, 1):
        order = np.random.default_rng(seed).permutation(len(L.pool))     # block i goes to order[i]
        moved = np.empty_like(L.pool)
        moved[order] = L.pool
        L.cache.pages.copy_(torch.from_numpy(moved.reshape(-1)))
        L.cache.page_table.copy_(torch.from_numpy(np.where(L.table < 0, -1, order[L.table]).astype(np.int32)))
        again, lse2 = decode(L, q)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert L.status() == 0


def test_decode_lengths_and_pages_out_of_bounds():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(8, [300, 200, 64], 4, 1, 128)
    q = O.bf16(L.g.standard_normal((3, 4, 128)))
    out, lse = decode(L, q)
    assert L.status() == 0
    L.cache.seq_len.copy_(i32([300, -5, 64]))
    got, got_lse = decode(L, q)
    assert L.status() == B.DEV_LENGTH and (got[1] == 0).all() and (got_lse[1] == -np.inf).all()
    assert (got[[0, 2]] == out[[0, 2]]).all()
    L.cache.dev_status.zero_()
    L.cache.seq_len.copy_(i32([10 ** 9, 200, 64]))
    got, _ = decode(L, q)
    assert L.status() == B.DEV_LENGTH and (got == out).all()     # clamped to max_len = 300
    L.cache.dev_status.zero_()
    L.cache.seq_len.copy_(i32([300, 200, 64]))
    for bad in (-1, L.cache.n_pages, 2 ** 31 - 1):
        table = L.table.copy()
        table[0, 3], table[2, :4] = bad, bad
        L.cache.page_table.copy_(torch.from_numpy(table))
        got, got_lse = decode(L, q)
        assert L.status() == B.DEV_PAGE_BOUNDS and (got[1] == out[1]).all()
        assert (got[2] == 0).all() and (got_lse[2] == -np.inf).all()
        keep = np.r_[0:48, 64:300]
        for h in range(4):
            want, _, _ = O.masked_attention(O.modified_scores(q[0, h:h + 1], L.k[0][keep, 0], 299), L.v[0][keep, 0])
            assert (np.abs(host(got)[0, h] - want[0]) <= HALF_BF16 * np.abs(want[0]) + 2.0 ** -12 * np.abs(L.v[0]).max()).all()
        L.cache.dev_status.zero_()


@pytest.mark.parametrize("hq", [8, 16])
def test_decode_nan_query_stays_in_its_head(hq):
    L = Layer(4, [700, 33], hq, 1, 128)
    q = O.bf16(L.g.standard_normal((2, hq, 128)))
    out, lse = decode(L, q)
    bad = q.copy()
    bad[0, 3, 5] = np.nan
    got, got_lse = decode(L, bad)
    assert got[0, 3].isnan().all() and got_lse[0, 3].isnan()
    keep = [h for h in range(hq) if h != 3]
    assert (got[0, keep] == out[0, keep]).all() and (got[1] == out[1]).all() and (got_lse[0, keep] == lse[0, keep]).all()


@pytest.mark.parametrize("scale_q,scale_v", [(2.0 ** 60, 1.0), (2.0 ** -60, 1.0), (1.0, 2.0 ** -18), (1.0, 2.0 ** 12), (30.0, 1.0)])
def test_decode_extreme_sizes(scale_q, scale_v):
    """Far scores (one key takes all, or all the same) and small and large values."""
    L = Layer(12, [600, 48], 4, 1, 128, fill=False)
    for b, n in enumerate(L.lens):
        L.k.append(L.put(b, np.arange(n), 0, O.bf16(L.g.standard_normal((n, 1, 128)))))
        L.v.append(L.put(b, np.arange(n), 1, O.bf16(scale_v * (L.g.standard_normal((n, 1, 128)) + 0.2))))
    L.upload()
    q = O.bf16(L.g.standard_normal((2, 4, 128)) * scale_q)
    out, lse = decode(L, q)
    assert L.status() == 0
    for b, n in enumerate(L.lens):
        for h in range(4):
            t = O.modified_scores(q[b, h:h + 1], L.k[b][:, 0], n - 1)
            top = np.sort(t[0])[::-1]
            want, _, want_lse = O.masked_attention(t, L.v[b][:, 0])
            # a score's error is 2^-21 of its terms' sum (2^-22 of it for each of two summands)
            err = 2.0 ** -21 * (np.abs(q[b, h]).sum() * np.abs(L.k[b]).max() * 2) / np.sqrt(128)
            if err > 0.01 and top[0] - top[1] < 40 + 2 * err:
                continue                              # two keys within the error: either may win
            near = HALF_BF16 * np.abs(want[0]) + (min(err, 0.01) * 2 + 2.0 ** -13) * np.abs(L.v[b]).max()
            assert (np.abs(host(out)[b, h] - want[0]) <= near).all()
            assert abs(host(lse)[b, h] - want_lse[0]) <= 2.0 ** -13 + err + 2.0 ** -22 * abs(want_lse[0])


@pytest.mark.parametrize("hq,d,form", [(4, 128, {}), (8, 64, {}), (16, 128, {}), (4, 64, dict(softcap=3.0)), (6, 128, dict(slopes=True))])
@pytest.mark.parametrize("power", [110, 118, 120])
def test_decode_queries_up_to_the_types_end(hq, d, form, power):
    """Queries of 2^112 to 2^122 whose scale makes ordinary scores of them."""
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(15, [700, 48, 1], hq, 1, d)
    q = O.bf16(L.g.standard_normal((3, hq, d)) * 2.0 ** power)
    scale = float(np.float32(2.0 ** -power / np.sqrt(d)))
    form = dict(form, scale=scale)
    if form.get("slopes"):
        form["slopes"] = 2.0 ** -np.arange(1.0, hq + 1)
    out, lse = decode(L, q, B.score_desc(scale, form.get("softcap", 0.0), 0, dev_f32(form["slopes"]) if "slopes" in form else None))
    assert L.status() == 0
    check_decode(L, q, out, lse, **form)


@pytest.mark.parametrize("hq,softcap", [(4, 0.0), (16, 0.0), (8, 30.0)])
def test_decode_largest_queries_on_keys_of_zeros(hq, softcap):
    """The largest finite channels of either sign: every score is 0, and the result the mean."""
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(16, [333, 5], hq, 1, 128, fill=False)
    for b, n in enumerate(L.lens):
        L.k.append(L.put(b, np.arange(n), 0, np.zeros((n, 1, 128))))
        L.v.append(L.put(b, np.arange(n), 1, O.bf16(L.g.standard_normal((n, 1, 128)))))
    L.upload()
    end = 255.0 * 2.0 ** 120
    q = np.where(L.g.random((2, hq, 128)) < 0.5, end, -end)
    q[:, 1, 3:] = 2.0 ** -100
    out, lse = decode(L, q, B.score_desc(0.0, softcap))
    check_decode(L, q, out, lse, softcap=softcap)


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("hq,d", [(4, 128), (9, 64)])
def test_decode_smallest_queries_with_scales_to_match(hq, d, softcap):
    """Queries of 2^-120 and a scale of 2^120: ordinary scores."""
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(18, [700, 48, 1], hq, 1, d)
    q = O.bf16(L.g.standard_normal((3, hq, d)))
    q = np.where(np.abs(q) < 2.0 ** -6, 0.0, q) * 2.0 ** -120
    scale = float(np.float32(2.0 ** 120 / np.sqrt(d)))
    tq = dev_bf16(q)
    assert (host(tq) == q).all()
    out, lse = decode(L, tq, B.score_desc(scale, softcap))
    check_decode(L, q, out, lse, scale=scale, softcap=softcap)


@pytest.mark.parametrize("ratio", [2.0 ** -14, 2.0 ** -20])
def test_decode_values_far_below_anothers_keep_their_bits(ratio):
    """A token of large values and no weight beside small ones that have all of it."""
    d, n = 128, 700
    L = Layer(13, [n], 4, 1, d, fill=False)
    k = L.g.standard_normal((n, 1, d))
    q = O.bf16(L.g.standard_normal((1, 4, d)))
    k[300, 0] = -8.0 * q[0].sum(0) / 2
    v = L.g.standard_normal((n, 1, d)) * 1000.0 * ratio
    v[300] = 1000.0 * L.g.standard_normal((1, d))
    L.k.append(L.put(0, np.arange(n), 0, O.bf16(k)))
    L.v.append(L.put(0, np.arange(n), 1, O.bf16(v)))
    L.upload()
    out, _ = decode(L, q)
    for h in range(4):
        t = O.modified_scores(q[0, h:h + 1], L.k[0][:, 0], n - 1)
        w, _, _ = O.masked_attention(t, np.eye(n))
        want = w[0] @ L.v[0][:, 0]
        size = w[0] @ np.abs(L.v[0][:, 0]).max(-1)
        # 2^-32 of the largest scale for each unit of weight and code, beside the other tokens' 2^-12
        near = HALF_BF16 * np.abs(want) + 2.0 ** -12 * size + 2.0 ** -32 * 255 * 8000.0 / 255
        assert w[0, 300] < 1e-9
        assert (np.abs(host(out)[0, h] - want) <= near).all()


def test_decode_strided_query_other_stream_and_graph():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    L = Layer(14, [1000, 64, 333], 8, 2, 64)
    q = O.bf16(L.g.standard_normal((3, 8, 64)))
    wide = torch.full((3, 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = dev_bf16(q)
    want, want_lse = decode(L, q)
    got, _ = decode(L, wide[:, 2:10])
    assert (got == want).all()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = [torch.zeros(B.oscar_decode_int8_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    B.oscar_decode_attention_int8(L.desc, wide[:, 2:10], out, ws[0], lse=lse, stream=side)
    side.synchronize()
    assert (out == want).all() and (lse == want_lse).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.oscar_decode_attention_int8(L.desc, wide[:, 2:10], out, ws[1], lse=lse)
    for _ in range(3):
        out.fill_(-7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert (out == want).all()


@pytest.mark.parametrize("hq,lens", [(4, [700, 33]), (16, [1500, 1])])
def test_decode_halves_join_by_their_logarithms(hq, lens):
    """The first and the last tokens decoded apart, and joined by the logarithms of the sums, are the whole."""
    d = 128
    L = Layer(31, lens, hq, 1, d)
    q = O.bf16(L.g.standard_normal((2, hq, d)))
    parts = []
    for cut in (0, 1):
        M = Layer(32, [max(0, n // 2 if cut == 0 else n - n // 2) for n in lens], hq, 1, d, fill=False)
        for b, n in enumerate(lens):
            rows = slice(0, n // 2) if cut == 0 else slice(n // 2, n)
            for which, x in ((0, L.k[b][rows]), (1, L.v[b][rows])):
                pos = np.arange(n)[rows]
                c, s, z = O.int8_load(L.pool, L.table[b, pos // 16], pos % 16, which, d)
                to = np.arange(len(pos))
                O.int8_store_rows(M.pool, M.table[b, to // 16], to % 16, which, c, s, z)
        M.upload()
        parts.append([host(x) for x in decode(M, q)])
    (o0, l0), (o1, l1) = parts
    top = np.maximum(l0, l1)
    w0, w1 = np.exp(l0 - top), np.exp(l1 - top)
    joined = (o0 * w0[..., None] + o1 * w1[..., None]) / (w0 + w1)[..., None]
    out, lse = decode(L, q)
    most = max(np.abs(v).max() for v in L.v)
    # three bf16 roundings and the bound of each decode
    assert (np.abs(joined - host(out)) <= HALF_BF16 * (np.abs(o0) + np.abs(o1) + np.abs(joined)) + 3 * 2.0 ** -12 * most).all()
    assert (np.abs(top + np.log(w0 + w1) - host(lse)) <= 2.0 ** -11).all()


def test_decodes_on_two_streams_at_once():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    layers = [Layer(41, [4000, 20, 900], 8, 2, 128), Layer(42, [2500, 1, 0, 3100], 20, 4, 64)]
    qs = [dev_bf16(L.g.standard_normal((len(L.lens), L.hq, L.d))) for L in layers]
    want = [decode(L, q)[0] for L, q in zip(layers, qs)]
    outs = [torch.zeros_like(w) for w in want]
    ws = [torch.zeros(B.oscar_decode_int8_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda") for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for L, q, o, w, s in zip(layers, qs, outs, ws, streams):
            B.oscar_decode_attention_int8(L.desc, q, o, w, stream=s)
    torch.cuda.synchronize()
    assert all((o == w).all() for o, w in zip(outs, want))


# ---------------------------------------------------------------- offsets beyond 32 bits

def test_pool_beyond_four_gigabytes():
    """Pages whose blocks lie beyond 2^32 bytes: appended, read back and decoded."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int8Cache
    d, hq, hk, n = 128, 4, 2, 100
    n_pages = (2 ** 32 + 2 ** 28) // (hk * O.int8_block_bytes(d))
    cache = Int8Cache(1, hq, hk, d, 7, n_pages)
    cache.page_table.copy_(i32([[n_pages - 1, 3, n_pages - 2, n_pages // 2 + 1, n_pages - 9, n_pages - 4, n_pages - 5]]))
    cache.seq_len.fill_(n)
    g = np.random.default_rng(1)
    q, k, v = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    req, pos = i32(np.zeros(n)), i32(np.arange(n))
    B.oscar_rope_append_int8(cache.desc(), None, None, None, dev_bf16(k), dev_bf16(v), req, pos, None)
    back = [torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.oscar_gather_int8(cache.desc(), req, pos, *back)
    out = torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(B.oscar_decode_int8_workspace_bytes(cache.desc()), dtype=torch.uint8, device="cuda")
    B.oscar_decode_attention_int8(cache.desc(), dev_bf16(q[-1:]), out, ws)
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == 0
    kv = [O.int8_values(*O.int8_quantize(x)) for x in (k, v)]
    for x, y in zip(back, kv):
        np.testing.assert_array_equal(host(x), O.bf16(y))
    for h in range(hq):
        want, _, _ = O.masked_attention(O.modified_scores(q[-1:, h], kv[0][:, h // 2], n - 1), kv[1][:, h // 2])
        assert (np.abs(host(out)[0, h] - want[0]) <= HALF_BF16 * np.abs(want[0]) + 2.0 ** -12 * np.abs(kv[1]).max()).all()


def test_rows_and_tables_beyond_two_billion_elements():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    d, n_pos = 128, 2 ** 24 + 70
    freq, _ = B.oscar_rope_frequencies(d, 1e6)
    table = torch.empty(n_pos, d, dtype=torch.float32, device="cuda")     # 2^31 entries and more
    B.oscar_rope_table(freq, table)
    rows = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(rows, (2, 3, d), (2 ** 31, d, 1))
    g = np.random.default_rng(2)
    data = O.bf16(g.standard_normal((2, 3, d)))
    x.copy_(dev_bf16(data))
    pos = np.array([n_pos - 1, 2 ** 24 + 1])
    B.oscar_norm_rope(None, B.rope_desc(table, d), x, None, i32(pos), x, None)
    torch.cuda.synchronize()
    cs = host(table[torch.from_numpy(pos).cuda()])
    want_cs = np.concatenate([O.rope_table(freq, int(p), 1) for p in pos])
    assert (np.abs(cs - want_cs) <= 2.0 ** -21 * np.abs(want_cs) + 2.0 ** -35).all()
    want, terms = rotated(data, None, cs, False)
    assert (np.abs(host(x) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms).all()


# ---------------------------------------------------------------- a run of them

def test_layer_run_prompt_then_tokens():
    """A table, two prompts appended and attended over what the cache holds, then tokens appended and decoded in a
    replayed graph, each against the oracle's own rows; the cache read back at the end."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    hq, hk, d, eps = 8, 2, 128, 1e-6
    prompts, steps = [70, 33], 5
    L = Layer(21, [p + steps for p in prompts], hq, hk, d, fill=False)
    g = L.g
    freq, magnitude = B.oscar_rope_frequencies(d, 1e4, "by_index", 4.0, 64.0)
    table = torch.empty(128, d, dtype=torch.float32, device="cuda")
    B.oscar_rope_table(freq, table, magnitude=magnitude)
    cs = host(table)
    wq, wk = (O.bf16(1 + 0.2 * g.standard_normal(d)) for _ in range(2))
    norm, rope = B.norm_desc(dev_bf16(wq), dev_bf16(wk), eps), B.rope_desc(table, d)
    n = sum(prompts)
    req = np.repeat([0, 1], prompts)
    pos = np.concatenate([np.arange(p) for p in prompts])
    q, k, v = (O.bf16(g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    qkv = dev_bf16(np.concatenate([q, k, v], 1))
    tq, tk, tv = qkv.split([hq, hk, hk], 1)
    q_rot = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    k_held, v_held = (torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.oscar_rope_append_int8(L.desc, norm, rope, tq, tk, tv, i32(req), i32(pos), q_rot, k_held=k_held, v_held=v_held)
    pd = B.prompt_desc(2, hq, hk, d, 70, 70, n, n)
    cu = i32([0, 70, n])
    out = torch.empty_like(q_rot)
    B.oscar_prompt_attention(pd, q_rot, k_held, v_held, cu, cu, out,
                             torch.empty(B.oscar_prompt_workspace_bytes(pd), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    # the cache holds what the append said, and that is the oracle's norm, rotation and codec within a step and a rounding
    hk_rows = [[], []]
    for which, held, x, w in ((0, k_held, k, wk), (1, v_held, v, None)):
        rows = O.rope(O.head_norm(x, w, eps), cs[pos], False) if which == 0 else x
        c, s, z = O.int8_quantize(O.bf16(rows))
        near = 0.51 * s.astype(float)[..., None] + 2.0 ** -7 * np.abs(rows)
        assert (np.abs(host(held) - rows) <= near).all()
        hk_rows[which] = [host(held)[req == b] for b in (0, 1)]
    group = hq // hk
    for b in (0, 1):
        rows = host(q_rot)[req == b]
        for h in range(hq):
            t = O.modified_scores(rows[:, h], hk_rows[0][b][:, h // group], 0)
            want, size, _ = O.masked_attention(t, hk_rows[1][b][:, h // group])
            assert (np.abs(host(out)[req == b][:, h] - want) <= HALF_BF16 * (np.abs(want) + size) + 2.0 ** -14).all()
    # tokens: one graph, replayed with new rows and places
    s_qkv = torch.zeros(2, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    s_pos, s_req = i32([0, 0]), i32([0, 1])
    s_q, s_out = (torch.zeros(2, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(B.oscar_decode_int8_workspace_bytes(L.desc), dtype=torch.uint8, device="cuda")

    def step():
        a, b, c = s_qkv.split([hq, hk, hk], 1)
        B.oscar_rope_append_int8(L.desc, norm, rope, a, b, c, s_req, s_pos, s_q)
        B.oscar_decode_attention_int8(L.desc, s_q, s_out, ws)
    L.cache.seq_len.copy_(i32([0, 0]))
    s_req.fill_(-1)
    step()                                            # (padding rows: nothing is written)
    s_req.copy_(i32([0, 1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        at = np.array([p + i for p in prompts])
        s_qkv.copy_(dev_bf16(g.standard_normal((2, hq + 2 * hk, d))))
        s_pos.copy_(i32(at)), L.cache.seq_len.copy_(i32(at + 1))
        graph.replay()
        torch.cuda.synchronize()
        for b in (0, 1):
            kk, vv = (torch.empty(at[b] + 1, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            B.oscar_gather_int8(L.desc, i32([b] * (at[b] + 1)), i32(np.arange(at[b] + 1)), kk, vv)
            pool = L.gpu_pool()
            p = np.arange(at[b] + 1)
            vals = [O.int8_values(*O.int8_load(pool, L.table[b, p // 16], p % 16, w, d)) for w in (0, 1)]
            assert (host(kk) == O.bf16(vals[0])).all() and (host(vv) == O.bf16(vals[1])).all()
            assert (host(kk)[:prompts[b]] == hk_rows[0][b]).all()
            new = O.rope(O.head_norm(host(s_qkv)[b:b + 1, hq:hq + hk], wk, eps), cs[at[b]:at[b] + 1], False)
            assert (np.abs(vals[0][-1] - new[0]) <= 2.0 ** -7 * np.abs(new).max()).all()
            for h in range(hq):
                t = O.modified_scores(host(s_q)[b, h:h + 1], vals[0][:, h // group], at[b])
                want, _, _ = O.masked_attention(t, vals[1][:, h // group])
                assert (np.abs(host(s_out)[b, h] - want[0]) <= HALF_BF16 * np.abs(want[0]) + 2.0 ** -12 * np.abs(vals[1]).max()).all()
    assert L.status() == 0


def test_rows_for_a_two_bit_layer():
    """A two-bit layer's step takes its keys from the norm and rotation: same bits as from rows rotated beforehand."""
    import torch
    import harness as H
    from bit_rotated_kv_split_gb300 import binding as B
    sc = H.Scenario(77, [700, 400], n_kv=2, g=4, cal=(256, 128))
    cache, _ = H.to_device(sc)
    g = np.random.default_rng(0)
    qkv = dev_bf16(g.standard_normal((2, 12, 128)))
    q, k, v = qkv.split([8, 2, 2], 1)
    table = torch.empty(1024, 128, dtype=torch.float32, device="cuda")
    B.oscar_rope_table(B.oscar_rope_frequencies(128, 1e6)[0], table)
    w = dev_bf16(1 + 0.1 * g.standard_normal(128))
    q_rot, k_rot = (torch.empty(2, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2))
    pos = i32([700, 400])
    B.oscar_norm_rope(B.norm_desc(w, w), B.rope_desc(table, 128), q, k, pos, q_rot, k_rot)
    src = i32([int(sc.recent_start[0]), 256 + int(sc.recent_start[1])])
    desc = cache.desc(int(sc.hist_len.max()) + 1)
    out = torch.empty(2, 8, 128, dtype=torch.float32, device="cuda")
    ws = torch.zeros(B.oscar_decode_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    hist = i32([int(x) for x in sc.hist_len])
    new_v = v.contiguous()
    ring = cache.recent_k.clone()
    B.oscar_quantize_append(desc, cache.recent_k.view(torch.uint16), cache.recent_v.view(torch.uint16), sc.B * 256, 2 * 128, src,
                            i32([0, 1]), hist, 2, new_k=k_rot.view(torch.uint16), new_v=new_v.view(torch.uint16))
    B.oscar_decode_attention(desc, q_rot.view(torch.uint16), out, ws)
    torch.cuda.synchronize()
    cs = host(table)
    want, terms = rotated(host(k), host(w), cs[[700, 400]], False)
    rows = cache.recent_k.reshape(-1, 2, 128)[src.long()]
    assert torch.equal(rows, k_rot)
    assert (np.abs(host(rows) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms).all()
    changed = (ring != cache.recent_k).reshape(-1, 256).any(1).nonzero().flatten().tolist()
    assert set(changed) <= set(src.tolist()) and torch.isfinite(out).all()
    assert int(cache.dev_status.item()) == 0


def test_normed_heads_into_a_four_bit_layer():
    """Heads normed and rotated by the one call, then appended without a rotation: the cache of those very rows."""
    import torch
    import test_gpu_int4 as F
    from bit_rotated_kv_split_gb300 import binding as B
    d, hq, hk, n = 128, 8, 2, 83
    L = F.Layer(23, [n], hq, hk, d, 64, 128, fill=False)
    q, k, v = (O.bf16(L.g.standard_normal((n, h, d))) for h in (hq, hk, hk))
    wq, wk = (O.bf16(1 + 0.2 * L.g.standard_normal(d)) for _ in range(2))
    cs = angles(n, d)
    tq, tk, tv = dev_bf16(np.concatenate([q, k, v], 1)).split([hq, hk, hk], 1)
    norm, rope = B.norm_desc(dev_bf16(wq), dev_bf16(wk)), B.rope_desc(dev_f32(cs), d)
    req, pos = i32(np.zeros(n)), i32(np.arange(n))
    k_rot = torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda")
    B.oscar_norm_rope(norm, rope, tq, tk, pos, tq, k_rot)                 # the queries in place
    B.oscar_rope_append_int4(L.desc, None, None, k_rot, tv, req, pos, None)
    torch.cuda.synchronize()
    for got, x, w in ((tq, q, wq), (k_rot, k, wk)):
        want, terms = rotated(x, w, cs, False)
        assert (np.abs(host(got) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -19 * terms).all()
    L.k.append(L.put(0, np.arange(n), 0, host(k_rot))), L.v.append(L.put(0, np.arange(n), 1, v))
    np.testing.assert_array_equal(L.gpu_pool(), L.pool)
    out = host(F.run_decode(L, tq[-1:]))
    ref, bound = F.weighted_ref(L, host(tq)[-1:])
    assert (np.abs(out - ref) <= bound).all() and L.status() == 0
