"""tq_sample against the float64 choice: settings, kinds of logits, odd sizes,
rows that are strided or not aligned, ends of the ranges."""
import math

import numpy as np
import pytest

from gpu_util import say
from sample_util import logits, sample

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# A double weight is off by some 2^-50 of it, a row's sums of up to 2^18 of them in
# steps of at least 2^-43 by up to 2^-26 in all: a choice nearer than that to another
# one is not compared (few are: see the count below).
NEAR = 2.0 ** -26


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def call(x, u, t=None, k=None, p=None, m=None, ws=None):
    import ternary_weight_base_amd as tq
    rows, vocab = x.shape
    xd = x if torch.is_tensor(x) else dev(x)
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), math.nan, device="cuda")
    f = lambda a, d: None if a is None else dev(np.asarray(a, dtype=d))
    if ws is None:
        ws = tq.sample_workspace(rows, vocab)
    tq.tq_sample(xd, f(u, np.float32), token, temperature=f(t, np.float32), top_k=f(k, np.int32), top_p=f(p, np.float32),
                 min_p=f(m, np.float32), logprob=lp, ws=ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert int(ws.count_nonzero()) == 0, "the workspace must be left zero"
    return token.cpu().numpy(), lp.cpu().numpy()


def verify(x, u, t=None, k=None, p=None, m=None, **more):
    """Compares every row whose choice is not nearer than NEAR to another; -> rows compared."""
    token, lp = call(x, u, t, k, p, m, **more)
    host = x.cpu().numpy() if torch.is_tensor(x) else x
    u = np.asarray(u, dtype=np.float32)
    n = 0
    for r in range(host.shape[0]):
        at = lambda a, d, v: v if a is None else d(a[r])
        f32 = lambda v: float(np.float32(v))
        want, want_lp, margin = sample(host[r], float(u[r]), at(t, f32, 1.0), at(k, int, 0), at(p, f32, 1.0), at(m, f32, 0.0))
        if margin <= NEAR:
            continue
        n += 1
        assert token[r] == want, (r, token[r], want, margin)
        # ln of a quotient that is off by up to 2^-25, rounded to fp32
        assert lp[r] == want_lp or abs(lp[r] - want_lp) <= 2.0 ** -24 * abs(want_lp) + 2.0 ** -24, (r, lp[r], want_lp)
    return n


SETTINGS = {"plain": {}, "temperature": {"t": (0.7, 1.3, 3.0)}, "k": {"k": (1, 2, 40, 300)}, "p": {"p": (0.1, 0.9, 0.99)},
            "m": {"m": (0.05, 0.5)}, "all": {"t": (0.8, 1.2), "k": (5, 50, 1000), "p": (0.5, 0.95), "m": (0.01, 0.1)},
            "mixed": {"t": (0.0, 0.6, 1.0, -1.0), "k": (0, 7, 1 << 30, -3), "p": (1.0, 0.6, 2.0), "m": (0.0, 0.2, -1.0)}}


def settings(rng, name, rows):
    return {n: rng.choice(v, rows) for n, v in SETTINGS[name].items()}


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("kind", ["usual", "steps", "masked", "one", "flat", "wide"])
@pytest.mark.parametrize("name", SETTINGS)
def test_settings(name, kind, dtype):
    say(f"sample {name} {kind} {dtype}")
    rng = np.random.default_rng(len(name) * 7 + len(kind))
    for rows, vocab in ((9, 5003), (3, 40000)):
        x = logits(rng, rows, vocab, kind, dtype)
        n = verify(x, rng.random(rows), **settings(rng, name, rows))
        assert n >= rows - 2 or kind in ("flat", "steps")  # (there a border between equal weights may fall on top_p's place)


@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 64, 65, 255, 4095, 4096, 4097, 8193, 131072, 150001])
def test_sizes(vocab):
    rng = np.random.default_rng(vocab)
    for dtype in ("float16", "float32"):
        for name in ("plain", "all", "mixed"):
            x = logits(rng, 5, vocab, "usual", dtype)
            verify(x, rng.random(5), **settings(rng, name, 5))


def test_largest_vocabulary():
    rng = np.random.default_rng(3)
    x = logits(rng, 2, 1 << 20, "usual", "float32")
    assert verify(x, rng.random(2), t=[1.0, 1.2], k=[0, 0], p=[0.9, 0.95]) >= 1
    assert verify(x, rng.random(2)) >= 1


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_large_k(dtype):
    """More tokens than are sorted: by their count, with top-p, and where fewer may come than k."""
    rng = np.random.default_rng(14)
    for kind, vocab in (("usual", 60000), ("masked", 60000), ("steps", 9000), ("flat", 9000)):
        x = logits(rng, 6, vocab, kind, dtype)
        k = [1024, 1025, 3000, 8000, vocab - 1, 5000]
        u = rng.random(6)
        assert verify(x, u, k=k) >= 5 or kind in ("steps", "flat")
        verify(x, u, k=k, m=[1e-3] * 6)
        verify(x, u, k=k, p=[0.3, 0.5, 0.9, 0.99, 0.7, 0.999], t=[0.3, 0.5, 1.0, 2.0, 5.0, 100.0])


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_steep_and_flat_temperatures(dtype):
    """The place of top-p from the first token to the bulk, in steps of few and of very many tokens."""
    rng = np.random.default_rng(15)
    x = logits(rng, 12, 70001, "usual", dtype)
    t = [0.01, 0.1, 0.3, 0.6, 1.0, 1.3, 2.0, 3.0, 5.0, 10.0, 100.0, 1e6]
    for p in (0.05, 0.5, 0.9, 0.99, 0.9999):
        assert verify(x, rng.random(12), t=t, p=[p] * 12) >= 11
        verify(x, rng.random(12), t=t, p=[p] * 12, m=[1e-4] * 12)
    for k in (1, 64, 1000):
        assert verify(x, rng.random(12), t=t, k=[k] * 12, p=[0.9] * 12) >= 11


def test_many_rows_of_more_than_one_segment():
    """More rows than a pass holds."""
    import ternary_weight_base_amd as tq
    rng = np.random.default_rng(16)
    rows, vocab = 1500, 4100
    assert tq.tq_sample_workspace_bytes(rows, vocab) < rows * 150000
    x = logits(rng, rows, vocab, "usual", "float16")
    u = rng.random(rows)
    token, lp = call(x, u, **settings(rng, "mixed", rows))
    assert token.min() >= 0
    pick = np.arange(0, rows, 37)
    rng = np.random.default_rng(17)
    s = settings(rng, "all", rows)
    token, _ = call(x, u, **s)
    for r in pick:
        want, _, margin = sample(x[r], float(np.float32(u[r])), *(float(np.float32(s[n][r])) if n != "k" else int(s[n][r]) for n in "tkpm"))
        assert margin <= NEAR or token[r] == want


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_strided_rows(dtype):
    rng = np.random.default_rng(4)
    for vocab, stride in ((5001, 5001), (5000, 5003), (4096, 5000), (10007, 10009)):
        x = logits(rng, 6, vocab, "usual", dtype)
        wide = torch.full((6, stride), math.inf, dtype=getattr(torch, dtype), device="cuda")
        wide[:, :vocab] = dev(x)
        assert verify(wide[:, :vocab], rng.random(6), **settings(rng, "all", 6)) >= 5


def test_rows_far_apart():
    """Rows 2^30 elements apart: byte offsets past 32 bits."""
    rng = np.random.default_rng(17)
    room = torch.empty((4, 1 << 30), dtype=torch.float16, device="cuda")
    for vocab in (1000, 9001):
        room[:, :vocab] = dev(logits(rng, 4, vocab, "usual", "float16"))
        room[:, vocab:vocab + 4096] = math.inf
        assert verify(room[:, :vocab], rng.random(4), **settings(rng, "all", 4)) >= 3


def test_the_place_of_u():
    """Each token's share of [0, 1): u at its borders and outside."""
    x = np.log(np.array([[1, 2, 4, 1]], dtype=np.float64)).astype(np.float32).repeat(9, 0)
    x[:, 0] = x[:, 3] = 0
    u = [0.0, 0.1249, 0.1251, 0.374, 0.376, 0.874, 0.876, 0.99999, 1.0]
    token, _ = call(x, u)
    assert token.tolist() == [0, 0, 1, 1, 2, 2, 3, 3, 3]
    token, _ = call(x, [-1.0, math.nan, 2.0, math.inf, 0.0, 0.0, 0.0, 0.0, 0.0], p=[1] * 4 + [0.0, -1.0, 0.4, math.nan, 0.6],
                    k=[0] * 4 + [2] * 5)
    # top-p of nothing, and up to the first, keep the largest alone; of 4 and 2, 0.6 does too, NaN limits nothing
    assert token.tolist() == [0, 0, 3, 3, 2, 2, 2, 1, 2]


def test_ties_go_to_the_lower_index():
    x = np.zeros((4, 6000), np.float32)
    x[:, 5000:] = 1.0
    x[3, 5000:] = -0.0
    token, lp = call(x, [0.999] * 4, t=[0.0, 1.0, 1.0, 1.0], k=[0, 1, 3, 5001])
    assert token.tolist() == [5000, 5000, 5002, 4995]  # the last row's zeros are all alike, the first 5001 stay
    assert lp[0] == 0 and lp[1] == 0 and abs(lp[2] + math.log(3)) < 1e-6 and abs(lp[3] + math.log(5001)) < 1e-5


def test_the_last_kept_token_weighs_little():
    """u of 1 and above: the last kept token, whatever its weight beside the others, on each way to it."""
    x = np.full((6, 9000), -math.inf, np.float32)
    x[:, 17] = 0.0
    x[:, 1000:2400] = -30.0
    x[:, 8999] = -45.0
    u = [1.0, 2.0, 1.0, 1.0, 1.0, 1.0 - 2.0 ** -24]
    for extra in ({}, {"k": [1402] * 6}, {"k": [1402, 1401, 1, 2, 1400, 900]}, {"p": [0.99] * 6}):
        assert verify(x, u, **extra) >= 5
    # (weights far below 1 are all near a min_p of their size: the tokens themselves; exp(-30) 9.4e-14, exp(-45) 2.9e-20)
    for extra, last in (({"k": [1402] * 6}, 8999), ({"k": [1000] * 6}, 1998), ({"m": [1e-30] * 6}, 8999), ({"k": [1402] * 6, "m": [1e-15] * 6}, 2399),
                        ({"k": [1000] * 6, "m": [1e-14] * 6}, 1998), ({"p": [0.99] * 6, "m": [1e-14] * 6}, 17)):
        token, _ = call(x, u, **extra)
        assert token[:5].tolist() == [last] * 5, (extra, token)


def test_ends_of_the_ranges():
    inf, nan, big = math.inf, math.nan, 3e38
    x = np.full((12, 5000), -inf, np.float32)
    x[1] = nan
    x[2, 4321] = -big                         # one token that may come
    x[3, [7, 4999]] = inf                     # infinite logits share everything
    x[3, 100:200] = 3
    x[4] = 0
    x[4, [3, 4]] = nan
    x[5, [10, 20]] = [big, -big]
    x[6, :] = 1.0
    x[7, [10, 4200]] = [1.0, 1.0 + 2.0 ** -23]
    x[8, [10, 4200]] = [5.0, 4.0]
    x[9, [1, 2, 3]] = [0.0, -1e-30, -2e-30]
    x[10, [10, 4200]] = [inf, 5.0]
    x[11] = np.linspace(-1e-3, 0, 5000)
    u = [0.5, 0.5, 0.5, 0.75, 0.0006, 0.9, 0.5, 0.9, 0.9, 0.5, 0.99, 0.5]
    t = [1.0, 1.0, 1e-6, 1.0, 1.0, 1e30, inf, 1e-30, 1e-30, 1.0, inf, 1e4]
    for extra in ({}, {"p": [0.95] * 12}, {"k": [3] * 12, "p": [0.999] * 12}, {"m": [1e-9] * 12}, {"k": [4000] * 12}):
        token, lp = call(x, u, t=t, **extra)
        assert token[0] == -1 and lp[0] == -inf and token[1] == -1 and lp[1] == -inf
        verify(x, u, t=t, **extra)


def test_rows_do_not_depend_on_each_other():
    rng = np.random.default_rng(8)
    x, u = logits(rng, 20, 30011, "usual", "float32"), rng.random(20)
    s = settings(rng, "mixed", 20)
    token, lp = call(x, u, **s)
    for r in (0, 7, 19):
        one, l1 = call(x[r:r + 1], u[r:r + 1], **{n: v[r:r + 1] for n, v in s.items()})
        assert one[0] == token[r] and l1[0] == lp[r]


def test_shares_of_many_draws():
    """100 000 draws over a small vocabulary: each token's count within six standard deviations."""
    rng = np.random.default_rng(9)
    n, vocab = 100000, 23
    x = rng.standard_normal(vocab).astype(np.float32)
    rows = dev(x).expand(n, vocab).contiguous()
    token, _ = call(rows, rng.random(n), k=np.full(n, 20))
    w = np.exp(x.astype(np.float64) - x.max())
    w[np.argsort(x)[:3]] = 0
    p = w / w.sum()
    c = np.bincount(token, minlength=vocab)
    assert np.all(np.abs(c - n * p) <= 6 * np.sqrt(n * p * (1 - p)) + 1e-9)


def test_captured_with_changing_logits():
    import ternary_weight_base_amd as tq
    rng = np.random.default_rng(10)
    rows, vocab = 5, 20001
    x = [dev(logits(rng, rows, vocab, k, "float32")) for k in ("usual", "steps", "masked", "flat", "usual")]
    s = {n: dev(np.asarray(v, np.int32 if n == "k" else np.float32)) for n, v in settings(rng, "all", rows).items()}
    u = dev(rng.random(rows).astype(np.float32))
    room, token, lp = x[0].clone(), torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    ws = tq.sample_workspace(rows, vocab)
    run = lambda a, b, c: tq.tq_sample(a, u, b, temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"], logprob=c, ws=ws)
    run(room, token, lp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(room, token, lp)
    for a in x:
        room.copy_(a)
        token.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        t2, l2 = torch.empty_like(token), torch.empty_like(lp)
        run(a, t2, l2)
        torch.cuda.synchronize()
        assert torch.equal(token, t2) and torch.equal(lp, l2)
