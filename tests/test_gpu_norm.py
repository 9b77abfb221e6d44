"""tq_residual_norm against its formula in 64 bits.  The kernel's sums and
products are doubles, so stored residuals and x are the correctly rounded
values but where a double lies within some 2^-50 of a rounding border: one
fp32 step (2^-23) is allowed there; the int8 codes are exact for that x."""
import numpy as np
import pytest

from gpu_util import dev, say
from kv_util import norm

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


SHAPES = [(1, 5120), (3, 1), (2, 3), (5, 64), (1, 127), (7, 1000), (2, 1030), (4, 4096), (1, 4100), (3, 8192), (2, 8193), (2, 17408),
          (1, 32768), (1, 32767), (700, 128)]
COMBOS = [("f4", "f4", True, "rows"), ("f2", "f4", True, "vector"), ("f4", "f2", False, "none"), ("f2", "f2", True, "strided")]


def _make(M, H, yt, rt, post, gate, seed):
    rng = np.random.default_rng(seed)
    y = (3 * rng.standard_normal((M, H))).astype(yt)
    res = (2 * rng.standard_normal((M, H))).astype(rt)
    pw = rng.uniform(0.5, 1.5, H).astype(np.float32) if post else None
    w = rng.uniform(0.5, 1.5, H).astype(np.float32)
    g = None
    if gate == "vector":
        g = rng.uniform(-1, 1, H).astype(yt)
    elif gate != "none":
        g = rng.uniform(-1, 1, (M, H)).astype(yt)
    return y, res, pw, w, g


def _close(got, want, what):
    """One step of the type at most, and hardly ever."""
    step = 2.0 ** (-23 if got.dtype == np.float32 else -10)
    tiny = 2.0 ** (-149 if got.dtype == np.float32 else -24)
    w = want.astype(np.float64)
    assert np.all(np.abs(got.astype(np.float64) - w) <= step * np.abs(w) + tiny), what
    assert np.mean(got != want) <= 1e-4 or np.sum(got != want) <= 1, (what, np.mean(got != want))


@pytest.mark.parametrize("combo", range(len(COMBOS)))
@pytest.mark.parametrize("M,H", SHAPES)
def test_residual_norm(M, H, combo):
    import ternary_weight_base_amd as tq
    yt, rt, post, gate = COMBOS[combo]
    say(f"norm {M}x{H} {COMBOS[combo]}")
    y, res, pw, w, g = _make(M, H, yt, rt, post, gate, M * 131 + H + combo)
    gd = None if g is None else dev(g)
    if gate == "strided":
        wide = torch.zeros((M, H + 12), dtype=gd.dtype, device="cuda")
        wide[:, :H] = gd
        gd = wide[:, :H]
        if H % 4 == 0 and M == 1:
            gd = gd.contiguous()
    out = torch.empty((M, H), dtype=torch.float32 if rt == "f4" else torch.float16, device="cuda")
    x32 = torch.empty((M, H), device="cuda")
    q, a = torch.empty((M, H), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    tq.tq_residual_norm(dev(y), dev(res), out, dev(w), x=x32, q=q, a_scale=a, post_w=None if pw is None else dev(pw), gate=gd,
                        res_scale=0.7, eps=1e-6)
    r, x = norm(y, res, np.dtype(rt), pw, g, 0.7, w, 1e-6)
    got_r = out.cpu().numpy()
    _close(got_r, r, "residual")
    # x is of the stored residual: stage by stage
    _, x = norm(None, got_r, None, None, None, 0, w, 1e-6)
    got_x = x32.cpu().numpy()
    _close(got_x, x.astype(np.float32), "x")
    # int8: the header's fp32 steps on the same x
    amax = np.abs(got_x).max(1)
    assert np.array_equal(a.cpu().numpy(), amax / np.float32(127))
    inv = np.float32(127) * (np.float32(1) / amax)
    assert np.array_equal(q.cpu().numpy(), np.clip(np.rint(got_x * inv[:, None]), -127, 127).astype(np.int8))
    if H % 128 == 0:
        # tq_quant_act divides once: its factor is within 2^-23 of this one (two roundings of 2^-24, one of its own),
        # which moves a product of at most 127 by 2^-16, so a code differs by one at most, where the
        # product is that near to a border: 2^-15 of them, 2^-14 allowed for (or one)
        q2, a2 = torch.empty_like(q), torch.empty_like(a)
        tq.tq_quant_act(x32, q2, a2)
        assert torch.equal(a, a2)
        off = (q.int() - q2.int()).abs()
        assert int(off.max()) <= 1 and int(off.sum()) <= max(1, M * H // 16384)
    # fp16 x, in place on the residual
    x16 = torch.empty((M, H), dtype=torch.float16, device="cuda")
    rd = dev(res)
    tq.tq_residual_norm(dev(y), rd, rd, dev(w), x=x16, post_w=None if pw is None else dev(pw), gate=gd, res_scale=0.7, eps=1e-6)
    assert np.array_equal(rd.cpu().numpy(), got_r)
    assert np.array_equal(x16.cpu().numpy(), got_x.astype(np.float16))


def test_first_block_zeros_and_no_weights():
    import ternary_weight_base_amd as tq
    say("norm without y, zero rows")
    rng = np.random.default_rng(3)
    res = rng.standard_normal((4, 640)).astype(np.float32)
    res[2] = 0
    x = torch.empty((4, 640), device="cuda")
    q = torch.full((4, 640), 5, dtype=torch.int8, device="cuda")
    a = torch.empty(4, device="cuda")
    tq.tq_residual_norm(None, dev(res), None, None, x=x, q=q, a_scale=a, eps=1e-5)
    _, want = norm(None, res, None, None, None, 0, None, 1e-5)
    _close(x.cpu().numpy(), want.astype(np.float32), "x")
    assert float(a[2]) == 0 and int(q[2].abs().max()) == 0 and int(q[1].abs().max()) == 127
    # eps 0 with a row of zeros: 0 / 0
    tq.tq_residual_norm(None, dev(res), None, None, x=x, eps=0.0)
    assert torch.isnan(x[2]).all() and torch.isfinite(x[[0, 1, 3]]).all()
    # only the addition
    out = torch.empty((4, 640), device="cuda")
    y = rng.standard_normal((4, 640)).astype(np.float32)
    tq.tq_residual_norm(dev(y), dev(res), out)
    assert np.array_equal(out.cpu().numpy(), (res.astype(np.float64) + y).astype(np.float32))


def test_nan_stays_in_its_row_and_large_values():
    import ternary_weight_base_amd as tq
    say("norm with nan and 1e38")
    rng = np.random.default_rng(4)
    y = rng.standard_normal((3, 512)).astype(np.float32)
    y[1, 7] = np.nan
    res = (rng.standard_normal((3, 512)) * 1e37).astype(np.float32)
    out, x = torch.empty((3, 512), device="cuda"), torch.empty((3, 512), device="cuda")
    w = np.ones(512, np.float32)
    tq.tq_residual_norm(dev(y), dev(res), out, dev(w), x=x, post_w=dev(w))
    assert torch.isnan(x[1]).all() and torch.isfinite(x[0]).all() and torch.isfinite(x[2]).all()
    r, want = norm(y[[0, 2]], res[[0, 2]], np.float32, w, None, 1.0, w, 1e-6)
    _close(x[[0, 2]].cpu().numpy(), want.astype(np.float32), "x")


def test_graph_replay():
    import ternary_weight_base_amd as tq
    say("norm in a graph")
    rng = np.random.default_rng(5)
    y, res = (torch.from_numpy(rng.standard_normal((2, 5120)).astype(np.float32)).cuda() for _ in range(2))
    out, w = torch.empty_like(res), torch.ones(5120, device="cuda")
    x = torch.empty((2, 5120), dtype=torch.float16, device="cuda")
    call = lambda: tq.tq_residual_norm(y, res, out, w, x=x, post_w=w, res_scale=0.5)
    call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.synchronize()
    for k in range(3):
        y.mul_(1.5)
        call()
        want = x.clone(), out.clone()
        x.zero_(), out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(out, want[1])


@pytest.mark.parametrize("M,H", [(3, 256), (2, 1001), (300, 2048)])
def test_smallest_values(M, H):
    """Rows whose largest element's reciprocal is past fp32, zeros among them."""
    import ternary_weight_base_amd as tq
    say(f"norm of tiny rows {M}x{H}")
    rng = np.random.default_rng(M)
    top = (2.0 ** rng.integers(-148, -95, (M, 1)))
    res = (rng.uniform(-1, 1, (M, H)) * top).astype(np.float32)
    res[:, ::5] = 0
    res[:, 1] = top[:, 0]
    x, q, a = torch.empty((M, H), device="cuda"), torch.empty((M, H), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    tq.tq_residual_norm(None, dev(res), None, x=x, q=q, a_scale=a, eps=1.0)
    got = x.cpu().numpy()
    assert np.array_equal(got, res)  # rms = 1 but for 2^-190
    up = got * np.float32(2.0 ** 100)
    inv = np.float32(127) * (np.float32(1) / np.abs(up).max(1))
    big = np.abs(got).max(1) >= 2.0 ** -100
    inv[big] = np.float32(127) * (np.float32(1) / np.abs(got[big]).max(1))
    up[big] = got[big]
    want = np.clip(np.rint(up * inv[:, None]), -127, 127).astype(np.int8)
    assert np.array_equal(q.cpu().numpy(), want) and np.all(want[:, ::5] == 0)
    assert np.array_equal(a.cpu().numpy(), np.abs(got).max(1) / np.float32(127))
