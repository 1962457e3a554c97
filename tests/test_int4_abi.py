"""CPU checks of the 4-bit layers' and the prompt attention's entry points:
block sizes, refusals before any launch, the binding's own checks and the
oracle's packing (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import oracle as O

FAKE = 1 << 20     # an aligned address that a refused call never touches


def _desc(**over):
    from bit_rotated_kv_split_gb300.binding import Int4Desc
    d = Int4Desc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim = 2, 8, 2, 128
    d.max_pages_per_seq, d.max_len, d.n_pages, d.tau_k, d.tau_v = 8, 100, 16, 10.0, 10.0
    d.pages = d.page_table = d.seq_len = FAKE
    for k, v in over.items():
        setattr(d, k, v)
    return d


def test_block_bytes_and_packing(built_lib):
    from bit_rotated_kv_split_gb300 import binding as B
    for d in (64, 128):
        for gk in (32, 64, 128):
            for gv in (32, 64, 128):
                want = O.int4_block_bytes(d, d // gk, d // gv) if max(gk, gv) <= d else 0
                assert B.oscar_int4_block_bytes(d, gk, gv) == want
        assert B.oscar_int4_block_bytes(d) == O.int4_block_bytes(d, 1, 1)
    for bad in ((96, 32, 32), (128, 16, 32), (128, 32, 256), (0, 0, 0), (128, -32, 32)):
        assert B.oscar_int4_block_bytes(*bad) == 0


@pytest.mark.parametrize("d,gk,gv", [(64, 32, 64), (128, 128, 32)])
def test_oracle_layout_covers_each_nibble_once(d, gk, gv):
    """Every nibble of a block belongs to one (K or V, slot, channel), and what is stored comes back."""
    ngk, ngv = d // gk, d // gv
    seen = set()
    for which in (0, 1):
        for slot in range(16):
            at, sh = O.int4_oracle._nibble(d, which, slot, np.arange(d))
            seen |= set(zip(at.tolist(), sh.tolist()))
    assert len(seen) == 2 * 16 * d and max(a for a, _ in seen) == 16 * d - 1
    g = np.random.default_rng(d)
    pool = g.integers(0, 256, (3, 2, O.int4_block_bytes(d, ngk, ngv))).astype(np.uint8)
    for which, ng in ((0, ngk), (1, ngv)):
        x = g.standard_normal((16, 2, d))
        c, s, z = O.int4_quantize(x, d // ng, 65504.0)
        assert np.abs(O.int4_values(c, s, z) - x).max() <= 0.51 * s.max() + 1e-3
        for slot in range(16):
            O.int4_store(pool, 1, slot, which, c[slot], s[slot], z[slot], ngk, ngv)
        c2, s2, z2 = O.int4_load(pool, [1] * 16, np.arange(16), which, d, ngk, ngv)
        np.testing.assert_array_equal(c, c2)
        np.testing.assert_array_equal(s, s2)
        np.testing.assert_array_equal(z, z2)
        rows = g.integers(0, 256, pool.shape).astype(np.uint8)
        O.int4_store_rows(rows, [2] * 16, np.arange(16), which, c, s, z, ngk, ngv)
        np.testing.assert_array_equal(O.int4_load(rows, [2] * 16, np.arange(16), which, d, ngk, ngv)[0], c)


BAD_CACHE = [
    (dict(batch=0), 1), (dict(n_q_heads=7), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=96), 1), (dict(head_dim=256), 1),
    (dict(max_pages_per_seq=0), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(max_len=-1), 1),
    (dict(max_len=129), 1), (dict(tau_k=0.0), 1), (dict(tau_v=float("nan")), 1), (dict(tau_v=1e6), 1),
    (dict(quant_group_k=16), 1), (dict(quant_group_v=256), 1), (dict(head_dim=64, quant_group_k=128), 1),
    (dict(pages=0), 1), (dict(page_table=0), 1), (dict(pages=FAKE + 64), 2), (dict(page_table=FAKE + 2), 2),
    (dict(dev_status=FAKE + 1), 2), (dict(batch=70000), 6),
]


def _append(B, d, rope=None, **over):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, req=FAKE, pos=FAKE, rp=None, n=3, qo=FAKE * 2, ko=None)
    a.update(over)
    return B.lib.oscar_rope_append_int4(ctypes.byref(d), None if rope is None else ctypes.byref(rope), a["q"], a["qs"],
                                        a["k"], a["ks"], a["v"], a["vs"], a["req"], a["pos"], a["rp"], a["n"], a["qo"],
                                        a["ko"], None)


def _gather(B, d, **over):
    a = dict(req=FAKE, pos=FAKE, n=3, k=FAKE, ks=256, v=FAKE, vs=256)
    a.update(over)
    return B.lib.oscar_gather_int4(ctypes.byref(d), a["req"], a["pos"], a["n"], a["k"], a["ks"], a["v"], a["vs"], None)


def _decode(B, d, score=None, size=1 << 40, **over):
    a = dict(q=FAKE, qs=1024, out=FAKE, ws=FAKE)
    a.update(over)
    n = ctypes.c_size_t(size)
    return B.lib.oscar_decode_attention_int4(ctypes.byref(d), None if score is None else ctypes.byref(score), a["q"],
                                             a["qs"], a["out"], a["ws"], ctypes.byref(n), None)


@pytest.mark.parametrize("over,status", BAD_CACHE)
def test_cache_descriptor_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    for call in (_append, _gather, _decode):
        assert call(B, _desc(**over)) == status, call.__name__


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(k=None), 1), (dict(v=None), 1), (dict(req=None), 1), (dict(pos=None), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(qs=1020), 1), (dict(qs=1028), 1), (dict(ks=255), 1), (dict(vs=128), 1),
    (dict(q=FAKE + 8), 2), (dict(k=FAKE + 2), 2), (dict(ko=FAKE + 4), 2), (dict(pos=FAKE + 1), 2), (dict(rp=FAKE + 2), 2),
    (dict(q=FAKE, qo=FAKE, qs=2048), 1), (dict(ko=FAKE, ks=512), 1),
])
def test_append_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _append(B, _desc(), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(rot_dim=8), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=144), 1), (dict(interleaved=2), 1),
    (dict(cos_sin=0), 1), (dict(n_positions=0), 1), (dict(cos_sin=FAKE + 4), 2),
])
def test_rope_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    r = B.RopeDesc()
    r.cos_sin, r.n_positions, r.rot_dim = FAKE, 100, 128
    for k, v in over.items():
        setattr(r, k, v)
    assert _append(B, _desc(), rope=r) == status
    assert _append(B, _desc(), rope=r, n=0) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(req=None), 1), (dict(pos=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(ks=248), 1), (dict(vs=260), 1), (dict(k=FAKE + 8), 2), (dict(req=FAKE + 2), 2),
])
def test_gather_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _gather(B, _desc(), **over) == status


BAD_SCORE = [dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(softcap=-1.0),
             dict(softcap=float("inf")), dict(window=-1), dict(reserved=1), dict(scale=3e38), dict(softcap=3e38),
             dict(scale=1e30, softcap=1e-30)]


@pytest.mark.parametrize("over", BAD_SCORE)
def test_score_refusals(built_lib, over):
    from bit_rotated_kv_split_gb300 import binding as B
    s = B.ScoreDesc()
    for k, v in over.items():
        setattr(s, k, v)
    assert _decode(B, _desc(), score=s) == 1
    assert _prompt(B, _pdesc(), score=s) == 1
    s = B.ScoreDesc()
    s.slopes = FAKE + 2
    assert _decode(B, _desc(), score=s) == 2 and _prompt(B, _pdesc(), score=s) == 2


def _pdesc(**over):
    from bit_rotated_kv_split_gb300.binding import PromptDesc
    d = PromptDesc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim = 2, 8, 2, 128
    d.max_q, d.max_k, d.causal, d.total_q, d.total_k = 10, 20, 1, 20, 40
    for k, v in over.items():
        setattr(d, k, v)
    return d


def _prompt(B, d, score=None, size=1 << 40, **over):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, cq=FAKE, ck=FAKE, pre=None, out=FAKE, lse=None, ws=FAKE)
    a.update(over)
    n = ctypes.c_size_t(size)
    return B.lib.oscar_prompt_attention(ctypes.byref(d), None if score is None else ctypes.byref(score), a["q"], a["qs"],
                                        a["k"], a["ks"], a["v"], a["vs"], a["cq"], a["ck"], a["pre"], a["out"], a["lse"],
                                        a["ws"], ctypes.byref(n), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), 1), (dict(batch=65536), 6), (dict(n_q_heads=9), 1), (dict(head_dim=32), 1), (dict(max_q=-1), 1),
    (dict(max_k=-1), 1), (dict(total_q=-1), 1), (dict(total_k=1 << 31), 1), (dict(causal=2), 1), (dict(reserved=3), 1),
])
def test_prompt_descriptor_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _prompt(B, _pdesc(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(cq=None), 1), (dict(ck=None), 1),
    (dict(qs=1016), 1), (dict(ks=252), 1), (dict(vs=260), 1), (dict(q=FAKE + 2), 2), (dict(out=FAKE + 8), 2),
    (dict(lse=FAKE + 2), 2), (dict(pre=FAKE + 1), 2), (dict(ws=FAKE + 16), 2), (dict(size=0), 3),
])
def test_prompt_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _prompt(B, _pdesc(), **over) == status


def test_prompt_without_queries_is_a_no_op(built_lib):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _prompt(B, _pdesc(max_q=0), q=None, out=None) == 0
    assert _prompt(B, _pdesc(total_q=0), q=None, out=None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(qs=1000), 1), (dict(q=FAKE + 8), 2), (dict(out=FAKE + 8), 2),
    (dict(ws=FAKE + 128), 2), (dict(size=0), 3),
])
def test_decode_refusals(built_lib, over, status):
    from bit_rotated_kv_split_gb300 import binding as B
    assert _decode(B, _desc(), **over) == status
    assert _decode(B, _desc(seq_len=0)) == 1
    assert _decode(B, _desc(n_q_heads=34)) == 6


def test_binding_checks():
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    with pytest.raises(ValueError):
        Int4Cache(1, 4, 1, 96, 1, 1, device="cpu")
    c = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
    desc = c.desc()
    assert desc.max_len == 64 and c.pages.numel() == 8 * 2 * O.int4_block_bytes(64, 1, 1)
    row = lambda n, h, d=64: torch.zeros(n, h, d, dtype=torch.bfloat16)   # noqa: E731
    idx = torch.zeros(3, dtype=torch.int32)
    bad = [dict(q=row(3, 8), k=row(2, 2)), dict(q=row(3, 8).float()), dict(k=row(3, 4)), dict(v=row(3, 2, 128)),
           dict(q_out=row(3, 9)), dict(k_out=row(3, 2).float()), dict(dst_req=idx.long()), dict(dst_pos=idx[:2]),
           dict(k=row(2, 3).transpose(0, 1).contiguous().transpose(0, 1)), dict(rope_pos=torch.zeros(6, dtype=torch.int32)[::2])]
    for over in bad:
        a = dict(q=row(3, 8), k=row(3, 2), v=row(3, 2), dst_req=idx, dst_pos=idx, q_out=row(3, 8), k_out=None, rope_pos=None)
        a.update(over)
        with pytest.raises(ValueError):
            B.oscar_rope_append_int4(desc, None, **a)
    with pytest.raises(ValueError):
        B.rope_desc(torch.zeros(4, 32), 64)
    with pytest.raises(ValueError):
        B.score_desc(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        B.oscar_decode_attention_int4(desc, row(2, 8), row(2, 8), torch.zeros(256, dtype=torch.uint8),
                                      score=B.score_desc(slopes=torch.zeros(4)))
    with pytest.raises(ValueError):
        B.oscar_decode_attention_int4(desc, row(1, 8), row(1, 8), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.oscar_gather_int4(desc, idx, idx, row(3, 2), row(2, 2))
    # rightly shaped, but not on a GPU: refused before the library sees a pointer
    with pytest.raises(ValueError, match="CUDA device"):
        B.oscar_rope_append_int4(desc, None, row(3, 8), row(3, 2), row(3, 2), idx, idx, row(3, 8))
    with pytest.raises(ValueError, match="CUDA device"):
        B.oscar_gather_int4(desc, idx, idx, row(3, 2), row(3, 2))
    with pytest.raises(ValueError, match="CUDA device"):
        B.oscar_decode_attention_int4(desc, row(2, 8), row(2, 8), torch.zeros(256, dtype=torch.uint8))
    pd = B.prompt_desc(1, 8, 2, 64, 3, 3, 3, 3)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.oscar_prompt_attention(pd, row(3, 8), row(4, 2), row(4, 2), cu, cu, row(3, 8), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.oscar_prompt_attention(pd, row(3, 8), row(3, 2), row(3, 2), cu[:1], cu, row(3, 8), torch.zeros(256, dtype=torch.uint8))


def test_binding_refuses_rows_of_other_types_and_descriptors_of_the_host():
    """fp16 has bf16's size; a table, slopes or pages in host memory must not reach a kernel."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    cache = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
    desc, idx = cache.desc(), torch.zeros(3, dtype=torch.int32)
    assert desc.keep is cache.pages

    def row(n, h, t=torch.bfloat16):
        return torch.zeros(n, h, 64, dtype=t)

    for over in (dict(q=row(3, 8, torch.float16)), dict(k=row(3, 2, torch.float16)), dict(q_out=row(3, 8, torch.float16)),
                 dict(k_out=row(3, 2, torch.float16))):
        a = dict(q=row(3, 8), k=row(3, 2), v=row(3, 2), dst_req=idx, dst_pos=idx, q_out=row(3, 8), k_out=None)
        a.update(over)
        with pytest.raises(ValueError, match="bfloat16"):
            B.oscar_rope_append_int4(desc, None, **a)
    with pytest.raises(ValueError, match="bfloat16"):
        B.oscar_gather_int4(desc, idx, idx, row(3, 2), row(3, 2, torch.float16))
    with pytest.raises(ValueError, match="bfloat16"):
        B.oscar_decode_attention_int4(desc, row(2, 8), row(2, 8, torch.float16), torch.zeros(256, dtype=torch.uint8))
    pd, cu = B.prompt_desc(1, 8, 2, 64, 3, 3, 3, 3), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="float32"):
        B.oscar_prompt_attention(pd, row(3, 8), row(3, 2), row(3, 2), cu, cu, row(3, 8), ws,
                                 lse=torch.zeros(3, 8, dtype=torch.int32))

    # of the tensors, only those that the descriptors point to are not on the device
    class OnDevice:
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    def dev(t):
        return OnDevice(t)

    a = [dev(row(3, 8)), dev(row(3, 2)), dev(row(3, 2)), dev(idx), dev(idx), dev(row(3, 8))]
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_rope_append_int4(desc, None, *a)
    desc.keep = dev(cache.pages)
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_rope_append_int4(desc, B.rope_desc(torch.zeros(4, 32), 32), *a)
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_decode_attention_int4(desc, dev(row(2, 8)), dev(row(2, 8)), dev(ws), score=B.score_desc(slopes=torch.zeros(8)))
    pd = B.prompt_desc(1, 8, 2, 64, 3, 3, 3, 3, dev_status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_prompt_attention(pd, dev(row(3, 8)), dev(row(3, 2)), dev(row(3, 2)), dev(cu), dev(cu), dev(row(3, 8)), dev(ws))


def test_cache_descriptor_keeps_its_tensors():
    """A descriptor that outlives its cache still points to live tables, lengths and status words."""
    import gc
    import weakref

    from bit_rotated_kv_split_gb300.cache import Int4Cache
    cache = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
    desc = cache.desc()
    refs = {name: weakref.ref(getattr(cache, name)) for name in ("pages", "page_table", "seq_len", "dev_status")}
    at = {name: getattr(cache, name).data_ptr() for name in refs}
    del cache
    gc.collect()
    for name, ref in refs.items():
        assert ref() is not None, name
        assert getattr(desc, name) == at[name] == ref().data_ptr()
    del desc
    gc.collect()
    assert all(ref() is None for ref in refs.values())


@pytest.mark.parametrize("which", [0, 1, 2])
def test_cache_descriptor_refuses_a_host_table(which):
    """A page table, lengths or a status word in host memory is refused before the library sees the pointer."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache

    class OnDevice:
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    cache = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
    desc, idx = cache.desc(), OnDevice(torch.zeros(3, dtype=torch.int32))
    rows = [OnDevice(torch.zeros(n, h, 64, dtype=torch.bfloat16)) for n, h in ((3, 8), (3, 2), (3, 2), (2, 8), (2, 8))]
    desc.keep = OnDevice(cache.pages)
    desc.keep_others = tuple(t if i == which else OnDevice(t) for i, t in enumerate(desc.keep_others))
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_rope_append_int4(desc, None, None, rows[1], rows[2], idx, idx, None)
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_gather_int4(desc, idx, idx, rows[1], rows[2])
    with pytest.raises(ValueError, match="one CUDA device"):
        B.oscar_decode_attention_int4(desc, rows[3], rows[4], OnDevice(torch.zeros(256, dtype=torch.uint8)))


def test_decode_refuses_lengths_whose_positions_pass_32_bits(built_lib):
    """Positions and page counts are 32-bit integers: max_len near 2^31 is refused, by the size query as well."""
    from bit_rotated_kv_split_gb300 import binding as B
    for n in (2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 512):
        d = _desc(max_pages_per_seq=1 << 27, max_len=n, batch=1, n_q_heads=1, n_kv_heads=1)
        assert _decode(B, d) == 6 and _decode(B, d, ws=None) == 6
    d = _desc(max_pages_per_seq=1 << 27, max_len=2 ** 31 - 513, batch=1, n_q_heads=1, n_kv_heads=1)
    assert _decode(B, d, ws=None) == 0


def test_binding_refuses_workspaces_that_are_not_contiguous():
    """numel of an expanded or strided view is not the memory behind it."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    desc = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu").desc()
    row = lambda n, h: torch.zeros(n, h, 64, dtype=torch.bfloat16)   # noqa: E731
    pd, cu = B.prompt_desc(1, 8, 2, 64, 3, 3, 3, 3), torch.zeros(2, dtype=torch.int32)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 24, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            B.oscar_decode_attention_int4(desc, row(2, 8), row(2, 8), ws)
        with pytest.raises(ValueError, match="workspace"):
            B.oscar_prompt_attention(pd, row(3, 8), row(3, 2), row(3, 2), cu, cu, row(3, 8), ws)


@pytest.mark.parametrize("over", [dict(batch=65535, max_q=2 ** 31 - 1, total_q=2 ** 31 - 1), dict(max_q=2 ** 31 - 1, n_q_heads=64, n_kv_heads=64)])
def test_prompt_refuses_grids_beyond_the_launch_limit(built_lib, over):
    """A valid description whose row blocks over all requests and heads are too many: unsupported, no CUDA error."""
    from bit_rotated_kv_split_gb300 import binding as B
    d = _pdesc(**over)
    assert _prompt(B, d, qs=64 * 128, ks=64 * 128, vs=64 * 128) == 6


def test_descriptors_refuse_numbers_beyond_32_bits():
    """ctypes cuts an integer to its field: a window of 2^32 + 5 would be one of 5."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="32-bit"):
            B.score_desc(window=n)
        with pytest.raises(ValueError, match="32-bit"):
            Int4Cache(1, 2, 1, 64, 4, 4, device="cpu").desc(n)
        for at in range(6):
            a = [1, 8, 2, 64, 3, 3]
            a[at] = n
            with pytest.raises(ValueError, match="32-bit"):
                B.prompt_desc(*a, 3, 3)
        with pytest.raises(ValueError):
            B.rope_desc(torch.zeros(4, 32), n)
    assert B.score_desc(window=2 ** 31 - 1).window == 2 ** 31 - 1


def test_cache_descriptor_refuses_tensors_that_do_not_fit():
    """A table, lengths, pages or a status word put in place of the cache's own have to be of its sizes and types."""
    import torch
    from bit_rotated_kv_split_gb300 import binding as B
    from bit_rotated_kv_split_gb300.cache import Int4Cache
    bad = dict(page_table=[torch.zeros(2, 3, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int64),
                           torch.zeros(4, 2, dtype=torch.int32).t(), torch.zeros(1, 1, dtype=torch.int32).expand(2, 4)],
               seq_len=[torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)[::2]],
               pages=[torch.zeros(100, dtype=torch.uint8)],
               dev_status=[torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int8)])
    for name, tensors in bad.items():
        for t in tensors:
            cache = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
            setattr(cache, name, t)
            with pytest.raises(ValueError, match=name):
                cache.desc()
    cache = Int4Cache(2, 8, 2, 64, 4, 8, device="cpu")
    cache.seq_len = torch.zeros(9, dtype=torch.int32)[3:5]
    assert cache.desc().seq_len == cache.seq_len.data_ptr()
    for t in bad["dev_status"]:
        with pytest.raises(ValueError, match="dev_status"):
            B.prompt_desc(1, 8, 2, 64, 3, 3, 3, 3, dev_status=t)
