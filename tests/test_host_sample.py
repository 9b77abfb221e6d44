"""Host-side tests of tq_sample: every argument error is reported before any
device work; the binding's checks; the float64 choice's own pins."""
import math

import numpy as np
import pytest

import ternary_weight_base_amd as tq
from sample_util import sample
from test_host_abi import FAKE, MIS, ODD

L = tq.lib
NULL, SHAPE, ALIGN, DTYPE, SIZE = -1, -2, -3, -6, -7


def _call(dt=0, rows=4, vocab=50000, x=FAKE, stride=50000, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, o=FAKE, lp=FAKE, ws=FAKE, wb=1 << 40):
    return L.tq_sample(dt, rows, vocab, x, stride, t, k, p, m, u, o, lp, ws, wb, None)


def test_sample_validates_on_host():
    for name in ("x", "u", "o"):
        assert _call(**{name: None}) == NULL, name
    assert _call(dt=2) == DTYPE and _call(dt=-1) == DTYPE
    for bad in ({"rows": 0}, {"rows": (1 << 20) + 1}, {"vocab": 0}, {"vocab": (1 << 20) + 1, "stride": 1 << 21}, {"stride": 49999},
                {"stride": (1 << 31) + 1}):
        assert _call(**bad) == SHAPE, bad
    for name in ("x", "ws"):
        assert _call(**{name: MIS}) == ALIGN, name
    for name in ("t", "k", "p", "m", "u", "o", "lp"):
        assert _call(**{name: ODD}) == ALIGN, name
    need = tq.tq_sample_workspace_bytes(4, 50000)
    if need:
        assert _call(wb=need - 1) == SIZE and _call(ws=None, wb=0) == NULL
    for bad in ((0, 50000), (4, 0), (4, (1 << 20) + 1)):
        assert tq.tq_sample_workspace_bytes(*bad) == 0


def test_binding_checks():
    torch = pytest.importorskip("torch")
    f, i = torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 40))
    for args, kw in (((x[0], f, i), {}), ((x, f[:2], i), {}), ((x, f, i[:1]), {}), ((x, f, f), {}), ((x, i, i), {}),
                     ((x, f, i), {"top_k": f}), ((x, f, i), {"temperature": i}), ((x, f, i), {"top_p": f[:2]}),
                     ((x, f, i), {"min_p": f.double()}), ((x, f, i), {"logprob": f.half()}), ((x.t(), f, i), {})):
        with pytest.raises(ValueError):
            tq.tq_sample(*args, **kw)


def test_reference_pins():
    x = np.log([1.0, 2.0, 4.0, 1.0])
    assert [sample(x, u)[0] for u in (0.0, 0.12, 0.13, 0.37, 0.38, 0.87, 0.88, 1.0)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert abs(sample(x, 0.2)[1] - math.log(0.25)) < 1e-12
    assert sample(x, 0.99, k=1)[0] == 2 and sample(x, 0.99, k=3)[0] == 2 and sample(x, 0.01, k=3)[0] == 0  # of the ties index 0 stays
    assert sample(x, 0.99, p=0.5)[0] == 2 and sample(x, 0.1, p=0.51)[0] == 1
    assert sample(x, 0.0, m=0.4)[0] == 1 and sample(x, 0.0, m=2.0)[0] == 2
    assert sample(x, 0.0, t=0.0)[0] == 2 and sample([math.nan, -math.inf], 0.5)[0] == -1
    assert abs(sample(x, 0.5, t=0.5)[1] - math.log(16 / 22)) < 1e-12
