"""Host-side tests of tq_kv_attn_shared: every argument error is reported before
any device work; the binding's checks; the workspace's bound."""
import pytest

import ternary_weight_base_amd as tq
from test_host_abi import FAKE, MIS, ODD

L = tq.lib
NULL, SHAPE, ALIGN, VALUE, SIZE = -1, -2, -3, -4, -7


def _call(rows=4, seqs=3, groups=2, hq=8, hkv=2, d=128, q=FAKE, qs=1024, cu=FAKE, kv=FAKE, cs=FAKE, pl=FAKE, tb=FAKE, mp=4, k=FAKE,
          v=FAKE, ks=FAKE, vs=FAKE, n=9, xp=640, xo=256, sc=0.1, o=FAKE, os=1024, ws=FAKE, wb=1 << 40):
    return L.tq_kv_attn_shared(rows, seqs, groups, hq, hkv, d, q, qs, cu, kv, cs, pl, tb, mp, k, v, ks, vs, n, xp, xo, sc, o, os, ws, wb, None)


def test_kv_attn_shared_validates_on_host():
    for name in ("q", "cu", "kv", "cs", "pl", "tb", "k", "v", "ks", "vs", "o"):
        assert _call(**{name: None}) == NULL, name
    for bad in ({"rows": 0}, {"seqs": 0}, {"groups": 0}, {"groups": (1 << 20) + 1}, {"hq": 9}, {"hkv": 0}, {"d": 80}, {"mp": 0}, {"n": 0}, {"qs": 1016},
                {"os": 1020}, {"xo": 0}, {"xp": -1}, {"qs": 1028}, {"xp": 1 << 31}, {"xp": 1 << 30, "xo": 1 << 30}):
        assert _call(**bad) == SHAPE, bad
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert _call(sc=bad) == VALUE, bad
    for name in ("q", "o", "k", "v", "ws"):
        assert _call(**{name: MIS}) == ALIGN, name
    for name in ("cu", "kv", "cs", "pl", "tb", "ks", "vs"):
        assert _call(**{name: ODD}) == ALIGN, name
    many = dict(rows=64, seqs=64, xp=16384, xo=300)  # two launches
    need = tq.tq_kv_attn_shared_workspace_bytes(64, 64, 2, 8, 2, 128, 16384, 300)
    assert need > tq.tq_kv_attn_workspace_bytes(64, 64, 8, 2, 128, 16684) > 0
    assert _call(**many, wb=need - 1) == SIZE and _call(**many, ws=None, wb=0) == NULL
    few = dict(rows=4, seqs=4, groups=1, xp=8192, xo=300)  # one, as tq_kv_attn
    need = tq.tq_kv_attn_shared_workspace_bytes(4, 4, 1, 8, 2, 128, 8192, 300)
    assert need == tq.tq_kv_attn_workspace_bytes(4, 4, 8, 2, 128, 8492) > 0
    assert _call(**few, wb=need - 1) == SIZE and _call(**few, ws=None, wb=0) == NULL
    for bad in ((0, 1, 1, 8, 2, 128, 64, 9), (1, 1, 0, 8, 2, 128, 64, 9), (1, 1, 1, 8, 3, 128, 64, 9), (1, 1, 1, 8, 2, 100, 64, 9),
                (1, 1, 1, 8, 2, 128, 64, 0), (1, 1, 1, 8, 2, 128, -1, 9)):
        assert tq.tq_kv_attn_shared_workspace_bytes(*bad) == 0


def test_lengths_at_the_end_of_64_bits():
    """Their sum is not taken before each is known to be small."""
    end = (1 << 63) - 1
    for xp, xo in ((end, 1), (end, end), (0, end), (end - 63, 256), (1 << 62, 1 << 62), ((1 << 31) - 1, 1), (1, (1 << 31) - 64)):
        assert _call(xp=xp, xo=xo) == SHAPE, (xp, xo)
        assert _call(rows=64, seqs=64, xp=xp, xo=xo) == SHAPE, (xp, xo)
        assert tq.tq_kv_attn_shared_workspace_bytes(64, 64, 2, 8, 2, 128, xp, xo) == 0, (xp, xo)


def test_workspace_is_bounded():
    most = max(tq.tq_kv_attn_shared_workspace_bytes(rows, seqs, groups, hq, hkv, dim, prefix, own)
               for rows in (1, 33, 130, 1040, 4096, 30000) for seqs in (1, 20, 64, 300) for groups in (1, 4, 20) if groups <= seqs
               for hq, hkv in ((8, 8), (64, 8), (5, 1)) for dim in (64, 128) for prefix in (0, 64, 5000, 131072) for own in (1, 1000, 20000))
    assert 0 < most <= 3 << 27


def test_binding_checks():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    f = lambda *s: torch.zeros(s)
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    ok = dict(q=h(4, 8, 64), cu_rows=i(4), kv_len=i(3), cu_seqs=i(3), prefix_len=i(2), page_table=i(3, 5), k_cache=u(9, 2, 64, 64),
              v_cache=u(9, 2, 64, 64), k_scale=f(9, 2), v_scale=f(9, 2), out=h(4, 8, 64), max_prefix_len=640, max_own_len=64)
    for name, bad in (("q", h(4, 512)), ("q", f(4, 8, 64)), ("out", h(4, 8, 32)), ("cu_rows", i(3)), ("cu_seqs", i(2)), ("cu_seqs", f(3)),
                      ("prefix_len", i(1, 2)), ("prefix_len", f(2)), ("kv_len", i(4)), ("k_scale", f(9, 3)), ("v_cache", u(9, 2, 64, 128))):
        with pytest.raises(ValueError):
            tq.tq_kv_attn_shared(**{**ok, name: bad})
