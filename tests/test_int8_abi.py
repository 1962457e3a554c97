"""CPU checks of the 8-bit layers' and the rotations' entry points: block
sizes, frequencies, refusals before any launch, the binding's own checks and the
oracle's packing (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest

import oracle as O

FAKE = 1 << 20     # an aligned address that a refused call never touches


def _desc(**over):
    from bit_rotated_kv_split_gb300.binding import Int8Desc
    d = Int8Desc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim = 2, 8, 2, 128
    d.max_pages_per_seq, d.max_len, d.n_pages, d.tau_k, d.tau_v = 8, 100, 16, 10.0, 10.0
    d.pages = d.page_table = d.seq_len = FAKE
    for k, v in over.items():
        setattr(d, k, v)
    return d


def test_block_bytes_and_packing(built_lib):
    from bit_rotated_kv_split_gb300 import binding as B
    for d in (64, 128):
        assert B.oscar_int8_block_bytes(d) == O.int8_block_bytes(d)
    for bad in (0, -64, 32, 96, 256):
        assert B.oscar_int8_block_bytes(bad) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_oracle_layout_covers_each_byte_once(d):
    seen = [int(b) for which in (0, 1) for slot in range(16) for b in O.int8_code_byte(d, which, slot, np.arange(d))]
    assert sorted(seen) == list(range(32 * d))
    # eight slots' chunks of the same channels lie in different 16-byte banks of 128 bytes
    for t0 in (0, 8):
        for c in range(d // 16):
            assert len({int(O.int8_code_byte(d, 0, t, 16 * c)) % 128 for t in range(t0, t0 + 8)}) == 8
    g = np.random.default_rng(d)
    pool = g.integers(0, 256, (3, 2, O.int8_block_bytes(d))).astype(np.uint8)
    for which in (0, 1):
        x = g.standard_normal((16, 2, d))
        c, s, z = O.int8_quantize(x)
        O.int8_store_rows(pool, [1] * 16, np.arange(16), which, c, s, z)
        for a, b in zip((c, s, z), O.int8_load(pool, [1] * 16, np.arange(16), which, d)):
            np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("shift", [0.0, 3.0, -500.0, 6e4, 1e-7])
@pytest.mark.parametrize("spread", [1.0, 1e-6, 200.0])
def test_codec_holds_every_value_within_half_a_step(shift, spread):
    x = O.bf16(np.clip(shift + spread * np.random.default_rng(3).standard_normal((200, 64)), -65000, 65000))
    c, s, z = O.int8_quantize(x)
    step = s.astype(np.float64)[:, None]
    assert (z.astype(np.float64) <= x.min(-1)).all()
    assert (np.abs(O.int8_values(c, s, z) - x) <= step / 2 + 1e-300).all()


SCALINGS = [dict(), dict(kind="linear", factor=4.0), dict(kind="base", factor=8.0),
            dict(kind="by_index", factor=4.0, original_len=32768.0), dict(kind="by_turns", factor=8.0, original_len=8192.0),
            dict(kind="by_index", factor=2.0, original_len=4096.0, turns_low=2.0, turns_high=16.0),
            dict(kind="by_turns", factor=32.0, original_len=100.0, turns_low=0.5, turns_high=3.0)]


@pytest.mark.parametrize("rot,theta", [(16, 1e4), (64, 1e4), (96, 5e5), (128, 1e6)])
@pytest.mark.parametrize("s", SCALINGS)
def test_frequencies_match_oracle(built_lib, rot, theta, s):
    from bit_rotated_kv_split_gb300 import binding as B
    got, magnitude = B.oscar_rope_frequencies(rot, theta, **s)
    kind = s.get("kind", "plain")
    low, high = s.get("turns_low", 0.0) or 1.0, s.get("turns_high", 0.0) or (32.0 if kind == "by_index" else 4.0)
    want, m = O.rope_frequencies(rot, theta, kind, s.get("factor", 1.0), s.get("original_len", 0.0), low, high)
    # powers and logarithms of a few ulps each, in ramps whose slope per index is at most 1
    np.testing.assert_allclose(got, want, rtol=1e-12)
    assert abs(magnitude - m) < 1e-15 * 4
    plain = B.oscar_rope_frequencies(rot, theta)[0]
    assert (got <= plain * (1 + 1e-12)).all() and (got >= plain / s.get("factor", 1.0) * (1 - 1e-12)).all()
    if kind == "base":
        assert abs(got[0] - 1) < 1e-15 and abs(got[-1] / plain[-1] * s["factor"] - 1) < 1e-12


@pytest.mark.parametrize("a", [
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=-16), dict(theta=1.0), dict(theta=float("inf")),
    dict(theta=float("nan")), dict(kind="linear", factor=0.5), dict(kind="linear", factor=float("nan")),
    dict(kind="base", factor=float("inf")), dict(kind="by_index", factor=2.0), dict(kind="by_turns", factor=2.0, original_len=0.5),
    dict(kind="by_turns", factor=2.0, original_len=100.0, turns_low=4.0, turns_high=4.0),
    dict(kind="by_index", factor=2.0, original_len=100.0, turns_low=-1.0, turns_high=4.0),
])
def test_frequencies_refusals(built_lib, a):
    from bit_rotated_kv_split_gb300 import binding as B
    with pytest.raises(B.OscarError) as e:
        B.oscar_rope_frequencies(**{**dict(rot_dim=64, theta=1e4), **a})
    assert e.value.status == 1


def test_frequencies_refuse_bad_structs(built_lib):
    from bit_rotated_kv_split_gb300 import binding as B
    out = np.empty(32)
    for s in (B.RopeScaling(5, 0, 1.0), B.RopeScaling(-1, 0, 1.0), B.RopeScaling(1, 1, 2.0)):
        assert B.lib.oscar_rope_frequencies(64, 1e4, ctypes.byref(s), out.ctypes.data, None) == 1
    assert B.lib.oscar_rope_frequencies(64, 1e4, None, None, None) == 1
    assert B.lib.oscar_rope_frequencies(64, 1e4, None, out.ctypes.data, None) == 0
    with pytest.raises(ValueError):
        B.oscar_rope_frequencies(64, 1e4, "cubic")


@pytest.mark.parametrize("a,status", [
    (dict(rot=8), 1), (dict(rot=144), 1), (dict(first=-1), 1), (dict(n=-1), 1), (dict(first=(1 << 40) + 1), 1),
    (dict(mag=float("nan")), 1), (dict(mag=1e300), 1), (dict(freq=7.0), 1), (dict(freq=-1e-3), 1), (dict(freq=float("nan")), 1),
    (dict(out=None), 1), (dict(out=FAKE + 8), 2), (dict(n=0, out=None), 0),
])
def test_table_refusals(built_lib, a, status):
    from bit_rotated_kv_split_gb300 import binding as B
    a = {**dict(rot=64, first=0, n=4, mag=1.0, freq=0.5, out=FAKE), **a}
    freq = np.full(72, 0.25)
    freq[3] = a["freq"]
    assert B.lib.oscar_rope_table(freq.ctypes.data, a["rot"], a["mag"], a["first"], a["n"], a["out"], None) == status
    assert B.lib.oscar_rope_table(None, 64, 1.0, 0, 4, FAKE, None) == 1


def _rope(**over):
    from bit_rotated_kv_split_gb300 import binding as B
    r = B.RopeDesc()
    r.cos_sin, r.n_positions, r.rot_dim = FAKE, 100, 128
    for k, v in over.items():
        setattr(r, k, v)
    return r


def _norm(**over):
    from bit_rotated_kv_split_gb300 import binding as B
    r = B.HeadNorm()
    r.q_weight = r.k_weight = FAKE
    r.eps = 1e-6
    for k, v in over.items():
        setattr(r, k, v)
    return r


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _rows(B, norm=None, rope=None, **over):
    a = dict(hq=8, hk=2, d=128, q=FAKE, qs=1024, k=FAKE * 3, ks=256, pos=FAKE, n=3, qo=FAKE * 2, qos=1024, ko=FAKE * 4, kos=256, st=None)
    a.update(over)
    return B.lib.oscar_norm_rope(a["hq"], a["hk"], a["d"], _ref(norm), _ref(rope), a["q"], a["qs"], a["k"], a["ks"], a["pos"],
                                 a["n"], a["qo"], a["qos"], a["ko"], a["kos"], a["st"], None)


def _append(B, d, norm=None, rope=None, **over):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, req=FAKE, pos=FAKE, rp=None, n=3, qo=FAKE * 2, ko=None, kh=None, vh=None)
    a.update(over)
    return B.lib.oscar_rope_append_int8(ctypes.byref(d), _ref(norm), _ref(rope), a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                        a["vs"], a["req"], a["pos"], a["rp"], a["n"], a["qo"], a["ko"], a["kh"], a["vh"], None)


def _gather(B, d, **over):
    a = dict(req=FAKE, pos=FAKE, n=3, k=FAKE, ks=256, v=FAKE, vs=256)
    a.update(over)
    return B.lib.oscar_gather_int8(ctypes.byref(d), a["req"], a["pos"], a["n"], a["k"], a["ks"], a["v"], a["vs"], None)


def _decode(B, d, score=None, size=1 << 40, **over):
    a = dict(q=FAKE, qs=1024, out=FAKE, lse=None, ws=FAKE)
    a.update(over)
    n = ctypes.c_size_t(size)
    return B.lib.oscar_decode_attention_int8(ctypes.byref(d), _ref(score), a["q"], a["qs"], a["out"], a["lse"], a["ws"],
                                             ctypes.byref(n), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), 1), (dict(n_q_heads=7), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=96), 1), (dict(head_dim=256), 1),
    (dict(max_pages_per_seq=0), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(max_len=-1), 1),
    (dict(max_len=129), 1), (dict(tau_k=0.0), 1), (dict(tau_v=float("nan")), 1), (dict(tau_v=1e6), 1),
    (dict(pages=0), 1), (dict(page_table=0), 1), (dict(pages=FAKE + 64), 2), (dict(page_table=FAKE + 2), 2),
    (dict(dev_status=FAKE + 1), 2), (dict(batch=70000), 6),
])
def test_cache_descriptor_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    for call in (_append, _gather, _decode):
        assert call(B, _desc(**over)) == status, call.__name__


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(k=None), 1), (dict(v=None), 1), (dict(req=None), 1), (dict(pos=None), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(qs=1020), 1), (dict(qs=1028), 1), (dict(ks=255), 1), (dict(vs=128), 1),
    (dict(q=FAKE + 8), 2), (dict(k=FAKE + 2), 2), (dict(ko=FAKE + 4), 2), (dict(pos=FAKE + 1), 2), (dict(rp=FAKE + 2), 2),
    (dict(kh=FAKE + 8), 2), (dict(vh=FAKE + 2), 2), (dict(qo=FAKE, qs=2048), 1), (dict(ko=FAKE, ks=512), 1),
    (dict(kh=FAKE, ks=512), 1), (dict(vh=FAKE, vs=512), 1), (dict(ko=FAKE * 5, kh=FAKE * 5), 1),
    (dict(kh=FAKE * 5, vh=FAKE * 5), 1), (dict(qo=FAKE * 5, vh=FAKE * 5), 1), (dict(v=FAKE * 3, kh=FAKE * 3), 1),
    (dict(k=FAKE * 3, vh=FAKE * 3), 1), (dict(k=FAKE * 3, qo=FAKE * 3), 1),
])
def test_append_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _append(B, _desc(), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(hq=0), 1), (dict(hk=0), 1), (dict(hq=70000), 1), (dict(d=96), 1), (dict(d=0), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(q=None, qo=None, k=None, ko=None), 1),
    (dict(pos=None), 1), (dict(qs=1016), 1), (dict(qs=1028), 1), (dict(qos=1016), 1), (dict(ks=128), 1), (dict(kos=252), 1),
    (dict(q=FAKE + 8), 2), (dict(qo=FAKE + 4), 2), (dict(k=FAKE + 2), 2), (dict(ko=FAKE + 8), 2), (dict(pos=FAKE + 2), 2),
    (dict(st=FAKE + 1), 2), (dict(qo=FAKE, qos=2048), 1), (dict(ko=FAKE * 3, kos=512), 1),
    (dict(qo=FAKE * 3), 1), (dict(ko=FAKE), 1), (dict(ko=FAKE * 2), 1),
])
def test_norm_rope_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _rows(B, _norm(), _rope(), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(rot_dim=8), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=144), 1), (dict(interleaved=2), 1),
    (dict(cos_sin=0), 1), (dict(n_positions=0), 1), (dict(cos_sin=FAKE + 4), 2),
])
def test_rope_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    for n in (0, 3):
        assert _append(B, _desc(), rope=_rope(**over), n=n) == status
        assert _rows(B, rope=_rope(**over), n=n) == status


@pytest.mark.parametrize("over,status", [
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(reserved=1), 1),
    (dict(q_weight=FAKE + 8), 2), (dict(k_weight=FAKE + 2), 2),
])
def test_norm_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    for n in (0, 3):
        assert _append(B, _desc(), norm=_norm(**over), n=n) == status
        assert _rows(B, norm=_norm(**over), n=n) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(req=None), 1), (dict(pos=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(ks=248), 1), (dict(vs=260), 1), (dict(k=FAKE + 8), 2), (dict(req=FAKE + 2), 2),
])
def test_gather_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _gather(B, _desc(), **over) == status


def test_gather_refuses_one_place_for_keys_and_values(built_lib):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _gather(B, _desc(), k=FAKE * 2, v=FAKE * 2) == 1
    assert _gather(B, _desc(), k=FAKE * 2, v=FAKE * 2, n=0) == 0


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(qs=1000), 1), (dict(q=FAKE + 8), 2), (dict(out=FAKE + 8), 2),
    (dict(lse=FAKE + 2), 2), (dict(ws=FAKE + 128), 2), (dict(size=0), 3),
])
def test_decode_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _decode(B, _desc(), **over) == status
    assert _decode(B, _desc(seq_len=0)) == 1
    assert _decode(B, _desc(n_q_heads=34)) == 6
    assert _decode(B, _desc(max_pages_per_seq=1 << 27, max_len=2 ** 31 - 512)) == 6
    s = B.ScoreDesc()
    s.window = -1
    assert _decode(B, _desc(), score=s) == 1


def test_binding_checks(built_lib):
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int8Cache
    with pytest.raises(ValueError):
        Int8Cache(1, 4, 1, 96, 1, 1, device="cpu")
    c = Int8Cache(2, 8, 2, 64, 4, 8, device="cpu")
    desc = c.desc()
    assert desc.max_len == 64 and c.pages.numel() == 8 * 2 * O.int8_block_bytes(64)
    assert desc.keep is c.pages and len(desc.keep_others) == 3
    row = lambda n, h, d=64: torch.zeros(n, h, d, dtype=torch.bfloat16)   # noqa: E731
    idx = torch.zeros(3, dtype=torch.int32)
    good = dict(norm=None, rope=None, q=row(3, 8), k=row(3, 2), v=row(3, 2), dst_req=idx, dst_pos=idx, q_out=row(3, 8))
    for over in [dict(q=row(3, 8), k=row(2, 2)), dict(q=row(3, 8).float()), dict(q=row(3, 8).half()), dict(k=row(3, 4)),
                 dict(v=row(3, 2, 128)), dict(q_out=row(3, 9)), dict(k_out=row(3, 2).float()), dict(k_held=row(2, 2)),
                 dict(v_held=row(3, 2, 128)), dict(dst_req=idx.long()), dict(dst_pos=idx[:2]),
                 dict(norm=B.norm_desc(torch.zeros(128, dtype=torch.bfloat16))),
                 dict(rope_pos=torch.zeros(6, dtype=torch.int32)[::2])]:
        with pytest.raises(ValueError):
            B.oscar_rope_append_int8(desc, **{**good, **over})
    ok = dict(norm=None, rope=None, q=row(3, 8), k=row(3, 2), pos=idx, q_out=row(3, 8), k_out=row(3, 2))
    for over in [dict(q=row(2, 8)), dict(k=row(3, 2, 128)), dict(q_out=None), dict(k=None), dict(q_out=row(3, 9)),
                 dict(k_out=row(2, 2)), dict(pos=idx.long()), dict(pos=idx[:2]), dict(q=row(3, 8).float()),
                 dict(dev_status=torch.zeros(1, dtype=torch.int64)), dict(norm=B.norm_desc(k_weight=torch.zeros(32, dtype=torch.bfloat16)))]:
        with pytest.raises(ValueError):
            B.oscar_norm_rope(**{**ok, **over})
    for bad in (torch.zeros(64), torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16)[::2]):
        with pytest.raises(ValueError):
            B.norm_desc(q_weight=bad)
    with pytest.raises(ValueError):
        B.oscar_rope_table(np.zeros(16), torch.zeros(4, 64))
    with pytest.raises(ValueError):
        B.oscar_rope_table(np.zeros(16), torch.zeros(4, 32, dtype=torch.float64))
    ws = torch.zeros(256, dtype=torch.uint8)
    for over in [dict(q=row(1, 8)), dict(out=row(2, 4)), dict(lse=torch.zeros(2, 8, dtype=torch.float64)), dict(lse=torch.zeros(2, 4)),
                 dict(workspace=ws[::2]), dict(score=B.score_desc(slopes=torch.zeros(4)))]:
        with pytest.raises(ValueError):
            B.oscar_decode_attention_int8(desc, **{**dict(q=row(2, 8), out=row(2, 8), workspace=ws), **over})
    with pytest.raises(ValueError):
        B.oscar_gather_int8(desc, idx, idx, row(3, 2), row(2, 2))
    # rightly shaped, but not on a GPU: refused before the library sees a pointer
    for call in (lambda: B.oscar_rope_append_int8(desc, **good), lambda: B.oscar_norm_rope(**ok),
                 lambda: B.oscar_gather_int8(desc, idx, idx, row(3, 2), row(3, 2)),
                 lambda: B.oscar_decode_attention_int8(desc, row(2, 8), row(2, 8), ws),
                 lambda: B.oscar_rope_table(np.zeros(16), torch.zeros(4, 32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_oracle_table_agrees_with_plain_doubles():
    freq, _ = O.rope_frequencies(64, 1e4)
    t = O.rope_table(freq, 5, 20)
    a = np.arange(5, 25)[:, None] * freq
    np.testing.assert_allclose(t, np.concatenate([np.cos(a), np.sin(a)], 1), atol=1e-14)


@pytest.mark.parametrize("first", ["B.oscar_rope_table(np.zeros(16), torch.zeros(4, 32))",
                                   "B.oscar_gather_int8(B.Int8Desc(), None, None, torch.zeros(0, 0, 0), torch.zeros(0, 0, 0))"])
def test_the_first_call_of_a_process_leaves_the_fast_checks_on(built_lib, first):
    """Whatever the process calls first, the short checks of later calls know their types."""
    import subprocess
    import sys
    code = "\n".join(["import numpy as np, torch", "from bit_rotated_kv_split_gb300 import binding as B", "try:", "    " + first,
                      "except ValueError:", "    pass", "assert B._bf16 is torch.bfloat16 and B._i32 is torch.int32"])
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("first", [2 ** 64, 2 ** 63, -2 ** 63 - 1, 2 ** 64 + 5])
def test_table_refuses_positions_beyond_64_bits(built_lib, first):
    """ctypes would take them modulo 2^64, as other positions."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    with pytest.raises(ValueError, match="first"):
        B.oscar_rope_table(np.zeros(16), torch.zeros(4, 32), first=first)
