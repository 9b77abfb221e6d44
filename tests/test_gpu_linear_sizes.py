"""tq_linear_attn in chunks where the sizes of rows differ by far more than
fp16 holds: zeros, rows that a reset has made nothing of, large rows behind
small ones, states that a chunk forgets.  Against the recurrence in float64,
each row by what it sees itself."""
import math

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = math.inf
TYPES = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reach(c):
    """For each row and KV head R_t = 2^g_t R_{t-1} + max|k_t| max|v_t|, R from the
    start's largest element: a bound of the state, of what is not forgotten alone.
    -> [rows][hkv], {sequence: its last}"""
    hq, hkv, dim = c["heads"]
    rows = c["qkv"].shape[0]
    x = c["qkv"].double().reshape(rows, hq + 2 * hkv, dim).abs().amax(2)
    g = (c["decay"].double() / math.log(2)).clamp(max=0).expand(rows, hkv)
    out, last = torch.zeros_like(g), {}
    for s, start in enumerate(c["from"]):
        R = torch.zeros(hkv, dtype=torch.float64, device="cuda")
        if 0 <= start < c["states"].shape[0]:
            R = c["states"][start].double().abs().amax((1, 2))
        for r in range(c["cu"][s], c["cu"][s + 1]):
            R = torch.exp2(g[r]) * R + x[r, hq:hq + hkv] * x[r, hq + hkv:]
            out[r] = R
        last[s] = R
    return out, last


def verify(c, out, states, outputs=True):
    """Tolerances of the chunked form.  Relative to the magnitudes (sums of the terms'
    absolute values) as linear_util derives them, with the log2 decays of rows that
    keep something.  Beside them what lies below fp16's least step, 2^-24, half of
    which a rounding loses: factors are scaled so that each row's largest element is
    in 2^13 .. 2^14, and a row's weights so that a bound of them, up to 8 times R
    (two powers of two and a power of two between), is 2^14 for states and, by
    dim max|q| R times another 2, 2^15 for outputs.
    States: 2^-25 of 2^14, 8 times, in keys and values of 128 rows: 2^(-39 + 3 + 1 + 7)
    = 2^-28 R.  Outputs: weights 2^(-25 - 15 + 4 + 7) = 2^-29, queries, keys, values
    2^-38 each, the state before the chunk 2^-38: together below 2^-28 dim max|q| R."""
    from linear_util import U, linear, out_tolerance, state_tolerance
    hq, hkv, dim = c["heads"]
    cu, rows = c["cu"], c["qkv"].shape[0]
    ref, mag, left, _ = linear(c["qkv"], c["decay"], cu, c["from"], c["to"], c["states"], c["scale"], hq, hkv, dim)
    bound, last = reach(c)
    g = (c["decay"].double() / math.log(2)).clamp(max=0).expand(rows, hkv)
    g = torch.where(g > -1000, -g, 0)
    most_q = c["qkv"].double()[:, :hq * dim].reshape(rows, hkv, hq // hkv, dim).abs().amax(3)
    for s in range(len(c["from"])):
        a, b = cu[s], cu[s + 1]
        fall = g[a:b].sum(0)
        sh = (b - a, hkv, hq // hkv, dim)
        small = 2.0 ** -28 * dim * abs(c["scale"]) * (most_q[a:b] * bound[a:b, :, None])[..., None]
        r, got = ref[a:b].reshape(sh), out[a:b].double().reshape(sh)
        tol = out_tolerance(r, mag[a:b].reshape(sh), 0.0, b - a, fall.reshape(1, hkv, 1, 1), dim, True) + small
        err = (got - r).abs()
        # an infinity is any result from 65520 on, of its sign: right where one of them is within
        # the tolerance (where terms cancel, the reference itself may be small or of the other sign)
        err = torch.where(torch.isinf(got) & (65520 - got.sign() * r <= tol), 0, err)
        bad = ~(err <= tol) & outputs
        say(f"  outputs: {float((err / tol).nan_to_num(INF).max()):.3g} of the tolerance")
        assert not bool(bad.any()), f"row {int(bad.flatten(1).any(1).nonzero()[0])} of sequence {s}: {float((err / tol).max())} of the tolerance"
        if c["to"][s] not in left:
            continue
        S, M, _ = left[c["to"][s]]
        err = (states[c["to"][s]].double() - S).abs()
        relative = (440 + 4 * math.ceil((b - a) / 128) + 2 * fall[:, None, None]) * U * M
        assert bool((relative <= state_tolerance(M, b - a, fall[:, None, None], True)).all())
        tol = relative + 2.0 ** -28 * last[s][:, None, None]
        say(f"  state: {float((err / tol.clamp(min=1e-300)).nan_to_num(INF).max()):.3g} of the tolerance")
        assert bool((err <= tol).all()), f"state of sequence {s}: {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"


def make(heads, n, dtype, seed, size=1.0):
    from test_gpu_linear import make as m
    c = m(heads, n, TYPES[dtype], "rows", seed, size=size)
    c["from"] = [-1] * len(n)
    return c


def run(c, outputs=True):
    from test_gpu_linear import call
    verify(c, *call(c), outputs=outputs)


def part(c, which):
    hq, hkv, dim = c["heads"]
    return {"rows": slice(None), "queries": slice(0, hq * dim), "keys": slice(hq * dim, (hq + hkv) * dim),
            "values": slice((hq + hkv) * dim, None)}[which]


@pytest.mark.parametrize("which", ["rows", "keys", "values"])
@pytest.mark.parametrize("dtype,size", [("f16", 1e-4), ("f32", 1e-6), ("f32", 1e-9)])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=str)
def test_zeros_before_small_rows(heads, dtype, size, which):
    """Padded or gated rows: half a chunk of zeros."""
    say(f"zeros {heads} {dtype} {size} {which}")
    c = make(heads, [128, 200], dtype, seed=40, size=size)
    for first in (0, 128 + 128):
        c["qkv"][first:first + 64, part(c, which)] = 0
    run(c)


# (row, times): rows before the reset at 90 of a chunk, in its first half or its second
FORGOTTEN = {"one": [10], "second half": [70], "several": [0, 31, 32, 63, 64, 89]}


def forgotten(heads, dtype, times, rows, n=300):
    """The second chunk has rows `times` as large as the others, forgotten at its 90th."""
    c = make(heads, [n], dtype, seed=41)
    for r in rows:
        c["qkv"][128 + r, c["heads"][0] * heads[2]:] *= times
    c["decay"][128 + 90] = -INF
    return c


@pytest.mark.parametrize("rows", FORGOTTEN)
@pytest.mark.parametrize("dtype,times", [("f16", 12000.0), ("f32", 1e4), ("f32", 1e6), ("f32", 1e10), ("f32", 1e15)])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=str)
def test_states_behind_forgotten_rows(heads, dtype, times, rows):
    say(f"forgotten {heads} {dtype} {times} {rows}")
    # the state of the second chunk's end, and one that the third one is added to
    run(forgotten(heads, dtype, times, FORGOTTEN[rows], n=256), outputs=False)
    run(forgotten(heads, dtype, times, FORGOTTEN[rows]), outputs=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=str)
def test_states_of_rows_of_all_sizes(heads, dtype):
    """Keys and values each by their own power of two, decays that halve and more."""
    say(f"all sizes {heads} {dtype}")
    c = make(heads, [333], dtype, seed=42)
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    most = 10 if dtype == "f16" else 60
    for which in ("keys", "values"):
        e = torch.randint(-most, most + 1, (333, 1), generator=g, device="cuda")
        c["qkv"][:, part(c, which)] *= torch.exp2(e.float()).to(TYPES[dtype])
    c["decay"] *= 20
    run(c, outputs=False)


@pytest.mark.parametrize("decay", ["reset", "slow"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (1, 1, 128)], ids=str)
def test_outputs_behind_a_forgotten_state(heads, dtype, decay):
    """A start 2^70 to 2^120 times what the chunk's rows add, forgotten at a row or bit by bit."""
    say(f"forgotten state {heads} {dtype} {decay}")
    for e in (70, 90, 120):
        c = make(heads, [200, 17], dtype, seed=43)
        c["from"] = [0, 1]
        c["states"] *= 2.0 ** e
        if decay == "reset":
            c["decay"][40] = c["decay"][203] = -INF
        else:
            c["decay"] *= 10
            c["decay"] -= 1.5
        run(c)


@pytest.mark.parametrize("rows", FORGOTTEN)
@pytest.mark.parametrize("dtype,times", [("f16", 12000.0), ("f32", 1e4), ("f32", 1e6), ("f32", 1e10), ("f32", 1e15)])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (1, 1, 128)], ids=str)
def test_outputs_behind_forgotten_rows(heads, dtype, times, rows):
    say(f"forgotten, outputs {heads} {dtype} {times} {rows}")
    run(forgotten(heads, dtype, times, FORGOTTEN[rows]))


@pytest.mark.parametrize("which", ["keys", "values", "queries"])
@pytest.mark.parametrize("dtype,e", [("f16", 13), ("f32", 28), ("f32", 32), ("f32", 40), ("f32", 70)])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (1, 1, 128)], ids=str)
def test_outputs_before_a_large_row(heads, dtype, e, which):
    """A key, value or query 2^e as large at the end of the chunk, and in the middle of 32 rows."""
    say(f"before a large row {heads} {dtype} {e} {which}")
    c = make(heads, [300], dtype, seed=44)
    for r in (127, 128 + 77):
        c["qkv"][r, part(c, which)] *= 2.0 ** e
        c["decay"][r + 1] = -INF
    run(c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (1, 1, 128)], ids=str)
def test_outputs_of_rows_of_all_sizes(heads, dtype):
    """Queries, keys and values each by their own power of two, decays that halve and more."""
    say(f"all sizes, outputs {heads} {dtype}")
    for seed in (45, 46):
        c = make(heads, [333], dtype, seed=seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        most = 10 if dtype == "f16" else 36
        for which in ("queries", "keys", "values"):
            e = torch.randint(-most, most + 1, (333, 1), generator=g, device="cuda")
            c["qkv"][:, part(c, which)] *= torch.exp2(e.float()).to(TYPES[dtype])
        c["decay"] *= 20
        c["scale"] *= 2.0 ** (-most // 2)
        run(c)


def test_small_rows_of_fp32():
    """Keys near fp32's least normal numbers, values (or queries) that make up for them."""
    for heads in ((4, 2, 128), (2, 2, 64)):
        c = make(heads, [200], "f32", seed=47)
        c["qkv"][:, part(c, "keys")] *= 2.0 ** -115
        c["qkv"][:, part(c, "values")] *= 2.0 ** 100
        c["qkv"][:, part(c, "queries")] *= 2.0 ** 15
        run(c)
        c["qkv"][:, part(c, "keys")] *= 2.0 ** 115
        c["qkv"][:, part(c, "queries")] *= 2.0 ** -130
        run(c)


@pytest.mark.parametrize("n", [128, 1500])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(2, 2, 128), (2, 2, 64)], ids=str)
def test_states_have_fp32s_accuracy(heads, dtype, n):
    """Root mean squares over a state, of terms of either sign, relative to the
    state's: a factor of two terms is off by up to 2^-23 evenly (2^-23.8 in the mean
    square, 2^-23.3 for two factors), the product of the second terms, 2^-11 each,
    is not taken (2^-11.8 each: 2^-23.6), a weight is an exp2 within 2^-23, and 24
    steps of 16 products a chunk are added in fp32 (2^-24.8 of a partial sum, some
    0.7 of the whole, each: 2^-23).  Together sqrt(2^-46.6 + 2^-47.2 + 2 * 2^-46) =
    2^-22.2, where an fp32 product and sum of 128 rows has about 2^-23."""
    from linear_util import linear
    from test_gpu_linear import call
    c = make(heads, [n], dtype, seed=48)
    _, states = call(c)
    S = linear(c["qkv"], c["decay"], c["cu"], c["from"], c["to"], c["states"], c["scale"], *heads)[2][c["to"][0]][0]
    got = float((states[c["to"][0]].double() - S).norm() / S.norm())
    say(f"states {heads} {dtype} {n}: {got:.3g}")
    assert got <= 2.0 ** -22


@pytest.mark.parametrize("dtype,size", [("f32", 1e-9), ("f16", 1e-4)])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64)], ids=str)
def test_what_strong_decays_leave_of_a_large_state(heads, dtype, size):
    """Decays of a chunk, or of eight, below fp32's least number, and what they leave is still the largest part."""
    say(f"large state decays {heads} {dtype}")
    for n, decay in (([128], -0.85), ([140], -0.85), ([1500], -0.1), ([1025, 40], -0.1), ([40, 77], -2.0)):
        c = make(heads, n, dtype, seed=49, size=size)
        c["from"] = list(range(len(n)))
        c["to"] = [len(n) + i for i in range(len(n))]
        c["states"] *= 2.0 ** 120 / size ** 2
        c["states"].clamp_(-2.0 ** 123, 2.0 ** 123)
        c["decay"] = torch.full_like(c["decay"], decay)
        run(c)


@pytest.mark.parametrize("n", [400, 1300])
def test_sizes_whose_sum_passes_fp32(n):
    """Elements of a state near fp32's largest, in different places: their sum, a bound of the state, is
    infinite, and is forgotten with them at a reset."""
    say(f"sum passes fp32 {n}")
    c = make((1, 1, 64), [n], "f32", seed=50)
    c["from"] = [0]
    c["states"][0, 0, 0, 0] = 3e38
    c["qkv"][:, 65:66] = 0   # nothing else is added there
    c["qkv"][5, 64:] = 0
    c["qkv"][5, 64 + 1], c["qkv"][5, 128 + 1] = 1e19, 2e19
    c["decay"][:] = 0
    c["decay"][128 + 40] = -INF
    run(c)
