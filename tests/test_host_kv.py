"""Host-side tests of the cache, attention and norm calls: every argument
error is reported before any device work; the rope table; the references'
own pins."""
import numpy as np
import pytest

import kv_plans
import ternary_weight_base_amd as tq
from kv_util import Cache, attention, rotate, scale_for
from test_host_abi import FAKE, MIS, ODD

L = tq.lib
NULL, SHAPE, ALIGN, VALUE, DTYPE, SIZE = -1, -2, -3, -4, -6, -7


def test_rope_table():
    t = tq.tq_rope_table(131072, 64, 1e6)
    i = np.arange(32)
    for p in (0, 1, 777, 131071):
        a = p * 1e6 ** (-2.0 * i / 64)
        # the angle in double is off by at most a few 2^-53 of it, far below half an fp32 step
        assert np.allclose(t[p, 0], np.cos(a), rtol=0, atol=2.0 ** -24) and np.allclose(t[p, 1], np.sin(a), rtol=0, atol=2.0 ** -24)
    buf = np.zeros(8, np.float32).ctypes.data
    assert L.tq_rope_table(1, 8, 1e4, None) == NULL
    for positions, rot in ((0, 8), (1, 0), (1, 12), (1, 136), (-3, 8)):
        assert L.tq_rope_table(positions, rot, 1e4, buf) == SHAPE
    for base in (1.0, 0.0, -5.0, float("inf"), float("nan")):
        assert L.tq_rope_table(1, 8, base, buf) == VALUE


def _append(dt=0, rows=4, seqs=2, hq=8, hkv=2, d=128, x=FAKE, stride=12 * 128, rope=FAKE, rr=100, rot=128, mode=0, cu=FAKE, kv=FAKE,
            tb=FAKE, mp=4, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n=9, q=FAKE):
    return L.tq_kv_append(dt, rows, seqs, hq, hkv, d, x, stride, rope, rr, rot, mode, cu, kv, tb, mp, k, v, ks, vs, n, q, None)


def test_kv_append_validates_on_host():
    for name in ("x", "rope", "cu", "kv", "tb", "k", "v", "ks", "vs"):
        assert _append(**{name: None}) == NULL, name
    assert _append(dt=2) == DTYPE
    assert _append(mode=2) == VALUE
    for bad in ({"rows": 0}, {"rows": (1 << 24) + 1}, {"seqs": 0}, {"hq": 0}, {"hkv": 0}, {"hq": 7}, {"d": 32}, {"d": 96}, {"d": 256},
                {"mp": 0}, {"n": 0}, {"rot": 12}, {"rot": 136}, {"rot": -8}, {"rr": 0}, {"stride": 12 * 128 - 8}, {"stride": 12 * 128 + 4},
                {"hq": 1 << 20}):
        assert _append(**bad) == SHAPE, bad
    for name in ("x", "rope", "k", "v", "q"):
        assert _append(**{name: MIS}) == ALIGN, name
    for name in ("cu", "kv", "tb", "ks", "vs"):
        assert _append(**{name: ODD}) == ALIGN, name


def _attn(rows=4, seqs=2, hq=8, hkv=2, d=128, q=FAKE, qs=1024, cu=FAKE, kv=FAKE, tb=FAKE, mp=4, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n=9,
          mk=256, sc=0.1, w=0, si=0, o=FAKE, os=1024, ws=FAKE, wb=1 << 40):
    return L.tq_kv_attn(rows, seqs, hq, hkv, d, q, qs, cu, kv, tb, mp, k, v, ks, vs, n, mk, sc, w, si, o, os, ws, wb, None)


def test_kv_attn_validates_on_host():
    for name in ("q", "cu", "kv", "tb", "k", "v", "ks", "vs", "o"):
        assert _attn(**{name: None}) == NULL, name
    for bad in ({"rows": 0}, {"seqs": 0}, {"hq": 9}, {"hkv": 0}, {"d": 80}, {"mp": 0}, {"n": 0}, {"qs": 1016}, {"os": 1020}, {"mk": 0},
                {"qs": 1028}, {"mk": 1 << 31}):
        assert _attn(**bad) == SHAPE, bad
    for bad in ({"w": -1}, {"si": -1}, {"sc": 0.0}, {"sc": -1.0}, {"sc": float("nan")}, {"sc": float("inf")}, {"w": 1 << 31}):
        assert _attn(**bad) == VALUE, bad
    for name in ("q", "o", "k", "v", "ws"):
        assert _attn(**{name: MIS}) == ALIGN, name
    for name in ("cu", "kv", "tb", "ks", "vs"):
        assert _attn(**{name: ODD}) == ALIGN, name
    need = tq.tq_kv_attn_workspace_bytes(4, 2, 8, 2, 128, 100000)
    assert need > 0
    assert _attn(mk=100000, wb=need - 1) == SIZE
    assert _attn(mk=100000, ws=None, wb=0) == NULL
    assert tq.tq_kv_attn_workspace_bytes(1, 1, 8, 2, 128, 64) == 0
    for bad in ((0, 1, 8, 2, 128, 64), (1, 0, 8, 2, 128, 64), (1, 1, 8, 3, 128, 64), (1, 1, 8, 2, 100, 64), (1, 1, 8, 2, 128, 0)):
        assert tq.tq_kv_attn_workspace_bytes(*bad) == 0


def test_kv_attn_workspace_is_bounded():
    most = max(tq.tq_kv_attn_workspace_bytes(rows, seqs, hq, hkv, dim, kv) for rows in (1, 7, 33, 130, 1040, 1041, 4096, 9000, 70000)
               for seqs in (1, 2, 20, 33, 64, 300) for hq, hkv in ((8, 8), (64, 8), (16, 2), (5, 1), (32, 32)) for dim in (64, 128)
               for kv in (1, 1024, 1025, 5000, 12288, 12289, 131072, 1 << 30))
    assert 0 < most <= 1 << 27
    assert tq.tq_kv_attn_workspace_bytes(1040, 33, 64, 8, 128, 13000) <= 1 << 27  # few rows left over among many places


def _norm(yt=1, rt=1, xt=1, m=2, h=640, y=FAKE, pw=FAKE, g=FAKE, gs=0, rs=1.0, r=FAKE, ro=FAKE, w=FAKE, eps=1e-6, x=FAKE, q=FAKE, a=FAKE):
    return L.tq_residual_norm(yt, rt, xt, m, h, y, pw, g, gs, rs, r, ro, w, eps, x, q, a, None)


def test_residual_norm_validates_on_host():
    assert _norm(r=None) == NULL
    assert _norm(a=None) == NULL          # codes need their scales
    assert _norm(ro=None) == NULL         # a block's output needs a residual to go to
    assert _norm(y=None) == NULL          # weights or gate of nothing
    assert _norm(y=None, pw=None) == NULL
    assert _norm(y=None, pw=None, g=None, ro=None, x=None, q=None) == NULL  # no output
    assert _norm(yt=2) == DTYPE and _norm(rt=-1) == DTYPE and _norm(xt=7) == DTYPE
    for bad in ({"m": 0}, {"h": 0}, {"h": 32769}, {"gs": 639}, {"gs": 642}):
        assert _norm(**bad) == SHAPE, bad
    for bad in ({"eps": -1.0}, {"eps": float("nan")}, {"rs": float("inf")}, {"rs": float("nan")}):
        assert _norm(**bad) == VALUE, bad
    for name in ("y", "pw", "g", "r", "ro", "w", "x", "q"):
        assert _norm(**{name: MIS}) == ALIGN, name
    assert _norm(a=ODD) == ALIGN


def test_kv_read_validates_on_host():
    f = lambda dt=0, n=2, h=2, d=64, p=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, num=4, o=FAKE: \
        L.tq_debug_kv_read(dt, n, h, d, p, k, v, ks, vs, num, o, None)
    for name in ("p", "k", "v", "ks", "vs", "o"):
        assert f(**{name: None}) == NULL, name
    assert f(dt=3) == DTYPE
    for bad in ({"n": 0}, {"h": 0}, {"d": 65}, {"num": 0}):
        assert f(**bad) == SHAPE, bad
    for name in ("k", "v", "o"):
        assert f(**{name: MIS}) == ALIGN, name
    for name in ("p", "ks", "vs"):
        assert f(**{name: ODD}) == ALIGN, name


def test_more_threads_than_a_launch_counts():
    assert _append(rows=(1 << 24) - 1, seqs=1) == SHAPE      # a workgroup of 256 threads a row
    assert _append(rows=(1 << 24) - 1, seqs=1 << 20, hq=32, hkv=32, stride=96 * 128) == SHAPE
    assert _attn(rows=1 << 20, seqs=1 << 20, hq=64, hkv=64, qs=8192, os=8192) == SHAPE  # a workgroup of 256 a row and head
    assert _norm(m=1 << 22) == SHAPE
    assert L.tq_debug_kv_read(0, 1 << 20, 8, 128, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 21, FAKE, None) == SHAPE


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("CPU tensors of a CPU-only process")
    i32 = torch.int32
    k, v = torch.zeros((3, 2, 64, 128), dtype=torch.uint8), torch.zeros((3, 2, 128, 64), dtype=torch.uint8)
    s, cu, kv, tb = torch.zeros((3, 2)), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((2, 4), dtype=i32)
    x, q = torch.zeros((4, 12 * 128)), torch.zeros((4, 8, 128), dtype=torch.float16)
    ok = dict(qkv=x, rope=None, cu_rows=cu, kv_len=kv, page_table=tb, k_cache=k, v_cache=v, k_scale=s, v_scale=s, q_out=q)
    for bad in ({"cu_rows": cu[:2]}, {"kv_len": kv.long()}, {"page_table": tb[:1]}, {"v_cache": k}, {"k_scale": s.half()},
                {"q_out": q.float()}, {"qkv": x[:, :-128]}, {"qkv": x.t()}, {"k_cache": k[0]}, {"page_table": tb.t().contiguous().t()}):
        with pytest.raises(ValueError):
            tq.tq_kv_append(**{**ok, **bad})
    at = dict(q=q, cu_rows=cu, kv_len=kv, page_table=tb, k_cache=k, v_cache=v, k_scale=s, v_scale=s, out=q, max_kv_len=64)
    for bad in ({"q": q.float()}, {"out": q[:3]}, {"q": q[..., :64], "out": q[..., :64]}, {"q": q.transpose(1, 2)}, {"v_scale": s[:2]}):
        with pytest.raises(ValueError):
            tq.tq_kv_attn(**{**at, **bad})
    r = torch.zeros((2, 640))
    for bad in ({"y": r[:1]}, {"x": r.t()}, {"res_out": r.half()}, {"pre_w": r}, {"gate": r[:1]}, {"gate": r[0].half()},
                {"q": r, "a_scale": r[0, :2]}, {"a_scale": r[0]}):
        with pytest.raises(ValueError):
            tq.tq_residual_norm(**{**dict(y=r, res=r, res_out=r), **bad})
    for bad in ({"post_w": r}, {"post_w": r[0].half()}, {"q": r.char(), "a_scale": r[:, 0]}, {"res": r.t().contiguous().t()},
                {"res_out": r.t().contiguous().t()}, {"y": r.half().t()}, {"x": r[:, :8]}):
        with pytest.raises(ValueError):
            tq.tq_residual_norm(**{**dict(y=r, res=r, res_out=r), **bad})
    rd = dict(pages=kv, k_cache=k, v_cache=v, k_scale=s, v_scale=s, values=torch.zeros((2, 2, 2, 64, 128)))
    for bad in ({"pages": kv.long()}, {"pages": tb}, {"k_cache": v}, {"v_cache": k}, {"k_scale": s.half()}, {"v_scale": s[:2]},
                {"values": torch.zeros((2, 2, 2, 64, 64))}, {"values": torch.zeros((2, 2, 2, 128, 64)).transpose(3, 4)}):
        with pytest.raises(ValueError):
            tq.tq_debug_kv_read(**{**rd, **bad})


def test_binding_refuses_host_memory_where_there_is_a_gpu(monkeypatch):
    """Before any call into the library: a kernel given a host address would fault."""
    torch = pytest.importorskip("torch")
    T = tq._Torch.get()
    monkeypatch.setattr(T, "available", lambda: True)
    monkeypatch.setattr(T, "device", lambda: 0)
    monkeypatch.setattr(T, "stream", lambda d: 0)

    def called(*a):
        raise AssertionError("the library was called")
    monkeypatch.setattr(tq, "lib", type("Lib", (), dict.fromkeys(("tq_kv_append", "tq_kv_attn", "tq_residual_norm", "tq_debug_kv_read"),
                                                                 staticmethod(called))))
    i32 = torch.int32
    k, v = torch.zeros((3, 2, 64, 128), dtype=torch.uint8), torch.zeros((3, 2, 128, 64), dtype=torch.uint8)
    s, cu, kv, tb = torch.zeros((3, 2)), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((2, 4), dtype=i32)
    q, r = torch.zeros((4, 8, 128), dtype=torch.float16), torch.zeros((2, 640))
    for call in (lambda: tq.tq_kv_append(torch.zeros((4, 12 * 128)), None, cu, kv, tb, k, v, s, s, q),
                 lambda: tq.tq_kv_attn(q, cu, kv, tb, k, v, s, s, q, 64),
                 lambda: tq.tq_residual_norm(r, r, r, x=r),
                 lambda: tq.tq_debug_kv_read(kv, k, v, s, s, torch.zeros((2, 2, 2, 64, 128)))):
        with pytest.raises(ValueError, match="current GPU"):
            call()


def test_references():
    """The references on cases worked by hand."""
    assert [scale_for(m) for m in (0.0, 1.0, 127.9, 128.0, 2.0 ** -130)] == [0.0, 2.0 ** -6, 1.0, 2.0, 2.0 ** -126]
    rope = np.zeros((2, 2, 2), np.float32)
    rope[1, 1] = 1  # position 1: a quarter turn of both pairs
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    assert rotate(x, 1, rope, 4, False).tolist() == [[-3.0, -4.0, 1.0, 2.0, 5.0]]
    assert rotate(x, 1, rope, 4, True).tolist() == [[-2.0, 1.0, -4.0, 3.0, 5.0]]
    c = Cache(1, 1, 2)
    c.put(0, 0, [[0.3, -0.3]], [[0.0, 0.0]])
    c.put(0, 1, [[1.0, -100.0]], [[0.0, 0.0]])
    scale, codes = c.codes(c.k, 0)
    assert scale[0] == 1.0 and codes[0].tolist() == [[128, 127]] and codes[1].tolist() == [[129, 28]]
    assert c.codes(c.v, 0)[0][0] == 0.0 and c.codes(c.v, 0)[1][1].tolist() == [[128, 128]]
    # two keys with the same score: the mean of their values; a row without keys: zeros
    k = np.full((1, 1, 64, 64), 128, np.uint8)
    v = np.full((1, 1, 64, 64), 128, np.uint8)
    v[0, 0, :, 1] = 130
    one = np.ones((1, 1), np.float32)
    q = np.ones((3, 1, 64), np.float16)
    out, _, _ = attention(q, [0, 3], np.array([2]), np.array([[0]], np.int32), k, v, one, one, 1.0, 0, 0)
    assert np.all(out[0] == 0) and np.all(out[1] == 0.5) and np.all(out[2] == 1.5)
    out, _, _ = attention(q, [0, 3], np.array([3]), np.array([[0]], np.int32), k, v, one, one, 1.0, 1, 0)
    assert np.all(out[1] == 2.5) and np.all(out[2] == 0.5)
    out, _, _ = attention(q, [0, 3], np.array([3]), np.array([[0]], np.int32), k, v, one, one, 1.0, 1, 1)
    assert np.all(out[1] == 1.5) and np.all(out[2] == 0.5)


def test_pages_of_all_units_are_counted_in_32_bits():
    """Where a few rows' keys are cut, the pages of all row tiles and KV heads,
    as many as the table is wide, must be fewer than 2^31 (128 units here)."""
    wide = dict(rows=4, seqs=2, hq=64, hkv=64, qs=8192, os=8192)
    assert tq.tq_kv_attn_workspace_bytes(4, 2, 64, 64, 128, 100000) > 0
    assert _attn(**wide, mk=100000, mp=1 << 24) == SHAPE
    assert _attn(rows=4, seqs=2, hq=64, hkv=32, qs=8192, os=8192, mk=100000, mp=1 << 25) == SHAPE


@pytest.mark.parametrize("name", kv_plans.PLANS)
def test_attention_plans(name):
    """The workspace of each call that tests/test_gpu_kv_attn_edges.py makes to
    take a plan."""
    hq, hkv, dim, lens, _, _, most, need = kv_plans.PLANS[name]
    assert tq.tq_kv_attn_workspace_bytes(sum(n for n, _ in lens), len(lens), hq, hkv, dim, most) == need
    assert max(t for _, t in lens) == most
