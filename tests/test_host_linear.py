"""Host-side tests of tq_linear_attn: every argument error is reported before
any device work; the binding's checks; the float64 recurrence's own pins."""
import math

import pytest

import ternary_weight_base_amd as tq
from test_host_abi import FAKE, MIS, ODD

L = tq.lib
NULL, SHAPE, ALIGN, VALUE, DTYPE, SIZE = -1, -2, -3, -4, -6, -7


def _call(dt=0, rows=4, seqs=2, hq=8, hkv=2, d=128, x=FAKE, stride=12 * 128, g=FAKE, gs=0, cu=FAKE, fr=FAKE, to=FAKE, st=FAKE, num=3,
          sc=0.1, o=FAKE, os=1024, ws=FAKE, wb=1 << 40):
    return L.tq_linear_attn(dt, rows, seqs, hq, hkv, d, x, stride, g, gs, cu, fr, to, st, num, sc, o, os, ws, wb, None)


def test_linear_attn_validates_on_host():
    for name in ("x", "g", "cu", "fr", "to", "st", "o"):
        assert _call(**{name: None}) == NULL, name
    assert _call(dt=2) == DTYPE and _call(dt=-1) == DTYPE
    for bad in ({"rows": 0}, {"rows": (1 << 24) + 1}, {"seqs": 0}, {"hq": 0}, {"hkv": 0}, {"hq": 7}, {"d": 32}, {"d": 96}, {"d": 256},
                {"num": 0}, {"num": 1 << 31}, {"stride": 12 * 128 - 8}, {"stride": 12 * 128 + 4}, {"gs": 1}, {"gs": -2}, {"os": 1016},
                {"os": 1028}, {"os": (1 << 22) + 8}, {"rows": 1 << 22, "hq": 256, "hkv": 256, "stride": 768 * 128, "os": 256 * 128}):
        assert _call(**bad) == SHAPE, bad
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert _call(sc=bad) == VALUE, bad
    for name in ("x", "st", "o", "ws"):
        assert _call(**{name: MIS}) == ALIGN, name
    for name in ("g", "cu", "fr", "to"):
        assert _call(**{name: ODD}) == ALIGN, name
    need = tq.tq_linear_attn_scratch_bytes(1000, 2, 8, 2, 128)
    assert need > 0
    assert _call(rows=1000, wb=need - 1) == SIZE
    assert _call(rows=1000, ws=None, wb=0) == NULL


def test_scratch():
    b = tq.tq_linear_attn_scratch_bytes
    assert b(1, 1, 8, 2, 128) == b(16, 1, 8, 2, 128) == b(160, 10, 8, 2, 128) == 0  # the recurrence needs none
    assert b(17, 1, 8, 2, 128) > 0
    for bad in ((0, 1, 8, 2, 128), (40, 0, 8, 2, 128), (40, 1, 8, 3, 128), (40, 1, 8, 2, 100)):
        assert b(*bad) == 0
    for rows in (17, 500, 4096, 1 << 20):
        for hq, hkv, d in ((64, 8, 128), (64, 64, 128), (16, 16, 64), (256, 256, 128)):
            if rows * hq < 1 << 30:
                assert b(rows, 1, hq, hkv, d) <= max((1 << 27) + 8 * hkv * d * d, 6 * hkv * d * d + 16 * hkv)


def test_binding_checks():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    def call(qkv=(6, 4 * 64), decay=(2,), cu=(3,), fr=(2,), states=(4, 2, 64, 64), out=(6, 4, 64), dt=torch.float16, st=torch.float32):
        tq.tq_linear_attn(torch.zeros(qkv, dtype=dt), torch.zeros(decay), torch.zeros(cu, **i32), torch.zeros(fr, **i32),
                          torch.zeros(2, **i32), torch.zeros(states, dtype=st), torch.zeros(out, dtype=torch.float16))
    ok = dict(qkv=(6, 8 * 64), out=(6, 4, 64))
    for bad in ({"qkv": (6, 7 * 64)}, {"decay": (3,)}, {"decay": (5, 2)}, {"cu": (4,)}, {"fr": (3,)}, {"states": (4, 2, 64, 32)},
                {"states": (2, 64, 64)}, {"out": (6, 256)}, {"st": torch.float64}):
        with pytest.raises(ValueError):
            call(**{**ok, **bad})


def test_reference_pins():
    """The recurrence against its closed form, by hand for two rows."""
    torch = pytest.importorskip("torch")
    from linear_util import linear
    dim = 64
    g = torch.Generator()
    g.manual_seed(1)
    qkv = torch.randn((2, 4 * dim), generator=g, dtype=torch.float64)
    states = torch.randn((1, 1, dim, dim), generator=g, dtype=torch.float64)
    decay = torch.tensor([[-0.25], [-1.5]])
    out, mag, left, fall = linear(qkv, decay, [0, 2], [0], [0], states, 0.5, 2, 1, dim)
    q, k, v = qkv[:, :2 * dim].view(2, 2, dim), qkv[:, 2 * dim:3 * dim], qkv[:, 3 * dim:]
    S1 = math.exp(-0.25) * states[0, 0] + torch.outer(k[0], v[0])
    S2 = math.exp(-1.5) * S1 + torch.outer(k[1], v[1])
    assert torch.allclose(out[0], 0.5 * q[0] @ S1, rtol=1e-12) and torch.allclose(out[1], 0.5 * q[1] @ S2, rtol=1e-12)
    assert torch.allclose(left[0][0][0], S2, rtol=1e-12) and bool((mag >= out.abs()).all())
    assert abs(float(fall[0]) - 1.75 / math.log(2)) < 1e-12
