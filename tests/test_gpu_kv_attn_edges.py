"""tq_kv_attn at the edges of what its arguments allow: pages that are not
there, weights far apart, the launch plans of each shape."""
import numpy as np
import pytest

from gpu_util import B3, dev, say, upload_blob, weights
from kv_plans import PLANS
from kv_util import PAGE, attention, attention_tolerance
from test_gpu_kv_attn import _check, _inputs, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# rows and lengths that the kernels for 16, 32 and 128 rows take
LENS = [[(1, 700)], [(50, 900)], [(1040, 2000)], [(1040, 1200), (300, 400), (1, 1)]]


@pytest.mark.parametrize("i", range(len(LENS)))
def test_missing_pages_beside_a_page_that_was_never_written(i):
    """Holes in the middle of a context, while page 0 of the pool, which no
    sequence holds, has whatever scales its memory had: the same output bits
    as with ordinary ones there."""
    lens = LENS[i]
    say(f"attention with holes and an unwritten page 0, {lens}")
    d = _inputs(np.random.default_rng(400 + i), 4, 2, 128, lens)
    table = d["table"]
    if (table == 0).any():  # page 0's place goes to a page that nobody holds
        table[table == 0] = next(p for p in range(len(d["ks"])) if not (table == p).any())
    table[0, 3], table[0, 7], table[0, 8] = -1, 1 << 20, -9
    clean = _run(d)
    _check(d, clean)
    for ks, vs in ((np.inf, np.inf), (2.0 ** -6, np.inf), (np.inf, 2.0 ** -6), (2.0 ** -6, 2.0 ** 122), (2.0 ** 100, 2.0 ** 127),
                   (np.nan, np.nan), (2.0 ** -6, np.nan), (-1.0, 2.0 ** 122), (0.0, 0.0), (2.0 ** -6, 2.0 ** -126)):
        d["ks"][0], d["vs"][0] = ks, vs
        assert np.array_equal(_run(d).view(np.uint16), clean.view(np.uint16)), (ks, vs)


# sequences' rows and lengths, max_kv_len: 16 rows whole and cut, 32 rows whole and cut, 128 rows
WEAK = [([(1, 900)], None), ([(1, 12000)], None), ([(5, 900)], None), ([(5, 12000)], None), ([(1040, 4096)], 20000)]


@pytest.mark.parametrize("first_page", [2.0 ** -4, 2.0 ** -14])
@pytest.mark.parametrize("gap", [16.0, 18.5])
@pytest.mark.parametrize("i", range(len(WEAK)))
def test_many_weak_keys_under_a_strong_one(i, gap, first_page):
    """A first token that draws all attention and has next to no value, under it
    keys of one sign that differ little: each weighs exp(-gap) of it, together
    they are the output.  Beside attention_tolerance's terms a weight below
    2^-25 of the row's largest may be off by 2^-36 of that (half of fp16's
    least step, the largest weight at 2^11 or above), times its value."""
    lens, most = WEAK[i]
    say(f"attention of weak keys, {lens}, gap {gap}, first page's scale {first_page}")
    rng = np.random.default_rng(500 + i)
    d = _inputs(rng, 4, 2, 128, lens)
    d["q"] = (1 + 0.02 * rng.standard_normal(d["q"].shape)).astype(np.float16)
    d["k"] = rng.integers(118, 138, d["k"].shape, dtype=np.uint8)
    d["v"] = rng.integers(160, 256, d["v"].shape, dtype=np.uint8)
    d["ks"][:], d["vs"][:] = 2.0 ** -6, 2.0 ** -4
    first = d["table"][0, 0]
    # score of code c against ones: 2^-6 (c - 127.5) 128 / sqrt(128)
    d["k"][first, :, 0] = round(127.5 + gap / (2.0 ** -6 * 128 ** 0.5))
    d["v"][first, :, :, 0] = rng.integers(127, 129, d["v"][first, :, :, 0].shape)
    d["vs"][first] = first_page
    ref, mag, dot = attention(d["q"], d["cu"], d["kv"], d["table"], d["k"], d["v"], d["ks"], d["vs"], 128 ** -0.5, 0, 0)
    keys = lens[0][1]
    tol = attention_tolerance(ref, mag, dot, keys, 128) + keys * 2.0 ** -36 * 128 * 2.0 ** -4
    err = np.abs(_run(d, max_kv=most).astype(np.float64) - ref)
    assert np.all(err <= tol), f"{np.max(err / tol)} of the tolerance, output {np.median(np.abs(ref))}"


@pytest.mark.parametrize("i", range(len(WEAK)))
def test_largest_scores(i):
    """The largest softmax_scale sum |q||k| that is taken, 2^20: such scores are
    off by several units, but the output stays a mean of values: within their
    range, off by the roundings of weights (2^-11, on both sums), of the sums
    (keys and keys / 64 rescalings, 2^-24 each, on both) and of the output (2^-11)."""
    lens, most = WEAK[i]
    say(f"attention of the largest scores, {lens}")
    rng = np.random.default_rng(600 + i)
    d = _inputs(rng, 4, 2, 128, lens)
    d["vs"][:] = 2.0 ** -7
    _, _, dot = attention(d["q"], d["cu"], d["kv"], d["table"], d["k"], d["v"], d["ks"], d["vs"], 1.0, 0, 0)
    bound = 127.5 * 2.0 ** -7 * (1 + 3 * 2.0 ** -11 + 2 * (lens[0][1] * 65 / 64 + 8) * 2.0 ** -24)
    for scale in (2.0 ** 20 / dot.max(), 2.0 ** 14 / dot.max()):
        got = _run(d, max_kv=most, scale=float(np.float32(scale * (1 - 2.0 ** -20)))).astype(np.float64)
        assert np.all(np.abs(got) <= bound), scale
        # and one key's score far above the rest: its value alone
        one = {**d, "k": d["k"].copy(), "q": np.abs(d["q"])}
        one["k"][d["table"][0, 0], :, 0] = 255
        one["k"][one["k"] > 200] = 200
        one["k"][d["table"][0, 0], :, 0] = 255
        one["ks"] = np.full_like(d["ks"], 2.0 ** -6)
        ref, mag, dot1 = attention(one["q"], d["cu"], d["kv"], d["table"], one["k"], d["v"], one["ks"], d["vs"], 1.0, 0, 0)
        s1 = float(np.float32(scale * dot.max() / dot1.max() * (1 - 2.0 ** -20)))
        ref, mag, _ = attention(one["q"], d["cu"], d["kv"], d["table"], one["k"], d["v"], one["ks"], d["vs"], s1, 0, 0)
        assert np.all(np.abs(_run(one, max_kv=most, scale=s1) - ref) <= 2.0 ** -9 * np.abs(ref) + 2.0 ** -25)


@pytest.mark.parametrize("rows,kv", [(1, 500), (200, 300)])
def test_page_table_of_any_width(rows, kv):
    """A table whose width times the row tiles passes 32 bits, in calls that
    keep no list of pages: as with a table of the pages that are used."""
    import ternary_weight_base_amd as tq
    say(f"attention with a wide page table, {rows} rows")
    d = _inputs(np.random.default_rng(700 + rows), 64, 64, 64, [(rows, kv), (rows, kv - 70)])
    want = _run(d)
    assert tq.tq_kv_attn_workspace_bytes(2 * rows, 2, 64, 64, 64, kv) == 0
    g = {k: dev(v) for k, v in d.items()}
    wide = torch.full((2, 1 << 25), -1, dtype=torch.int32, device="cuda")
    wide[:, :d["table"].shape[1]] = g["table"]
    out = torch.empty_like(g["q"])
    tq.tq_kv_attn(g["q"], g["cu"], g["kv"], wide, g["k"], g["v"], g["ks"], g["vs"], out, kv)
    assert np.array_equal(out.cpu().numpy().view(np.uint16), want.view(np.uint16))
    del wide
    torch.cuda.empty_cache()


def _reference(d, window, sinks):
    """kv_util.attention's three results for tables without holes, by float64
    products of whole heads on the CPU."""
    rows, hq, dim = d["q"].shape
    hkv, scale = d["ks"].shape[1], dim ** -0.5
    group = hq // hkv
    out, mag, dot = np.full((rows, hq, dim), np.nan), np.zeros((rows, hq, dim)), np.zeros((rows, hq))
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float64))
    for s, t in enumerate(d["kv"].tolist()):
        a, b = int(d["cu"][s]), int(d["cu"][s + 1])
        n = b - a
        if n == 0:
            continue
        ids = d["table"][s, :-(-t // PAGE)]
        pos, j = torch.arange(t - n, t)[:, None], torch.arange(t)[None]
        see = j <= pos
        if window:
            see = see & ((j > pos - window) | (j < sinks))
        see = see.repeat_interleave(group, 0)  # rows (token, head)
        for h in range(hkv):
            k = T((d["k"][ids, h].astype(np.float64) - 127.5) * d["ks"][ids, h][:, None, None]).reshape(-1, dim)[:t]
            v = T(((d["v"][ids, h].astype(np.float64) - 127.5) * d["vs"][ids, h][:, None, None]).transpose(0, 2, 1)).reshape(-1, dim)[:t]
            q = T(d["q"][a:b, h * group:(h + 1) * group]).reshape(-1, dim)
            z = torch.where(see, q @ k.T * scale, -torch.inf)
            w = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-1e300)) if t else z
            w = torch.nan_to_num(w / w.sum(1, keepdim=True))  # a row that sees nothing: zeros
            put = lambda x: x.reshape(n, group, dim).numpy()
            out[a:b, h * group:(h + 1) * group] = put(w @ v)
            mag[a:b, h * group:(h + 1) * group] = put(w @ v.abs())
            if t:
                dot[a:b, h * group:(h + 1) * group] = (q.abs() @ k.abs().T * scale * see).amax(1).reshape(n, group).numpy()
    return out, mag, dot


@pytest.mark.parametrize("name", PLANS)
def test_every_launch_plan(name):
    """Each plan against the 64-bit result, twice with the same bits, the
    workspace left zero."""
    import ternary_weight_base_amd as tq
    hq, hkv, dim, lens, window, sinks, most, need = PLANS[name]
    say(f"attention plan {name}: {hq}/{hkv} heads of {dim}, {len(lens)} sequences, {lens[:3]}, window {window}, sinks {sinks}")
    d = _inputs(np.random.default_rng(sum(map(ord, name))), hq, hkv, dim, lens)
    assert tq.tq_kv_attn_workspace_bytes(d["q"].shape[0], len(lens), hq, hkv, dim, most) == need
    got = _run(d, window, sinks, max_kv=most)
    assert np.array_equal(got.view(np.uint16), _run(d, window, sinks, max_kv=most).view(np.uint16))
    ref, mag, dot = _reference(d, window, sinks)
    tol = attention_tolerance(ref, mag, dot, most, dim)
    off = ~(np.abs(got.astype(np.float64) - ref) <= tol)
    assert not off.any(), f"{off.sum()} off, first at {np.argwhere(off)[0]}"


def test_infinite_queries_stay_in_their_row():
    """+inf, -inf, both and NaN in a query: every other row and head keeps its
    bits, also of other sequences."""
    say("attention of infinite queries")
    for i, (lens, most) in enumerate([([(2, 200), (1, 90)], None), ([(1, 5000), (3, 2000)], None), ([(80, 200)], None),
                                      ([(1040, 1100)], 20000), ([(300, 5000), (700, 900)], 20000)]):
        d = _inputs(np.random.default_rng(800 + i), 4, 2, 64, lens)
        clean = _run(d, max_kv=most)
        for at, bad in (((1, 2, 5), np.inf), ((0, 0, 63), -np.inf), ((len(d["q"]) - 1, 3, 0), np.nan)):
            d["q"][at] = bad
        d["q"][2, 1, :2] = np.inf, -np.inf
        got = _run(d, max_kv=most)
        hit = ((1, 2), (0, 0), (len(d["q"]) - 1, 3), (2, 1))
        assert np.isnan(got[hit[2]]).all() and np.isnan(got[hit[3]]).all()
        for at in hit:
            got[at] = clean[at]
        assert np.array_equal(got.view(np.uint16), clean.view(np.uint16)), lens


def test_workspace_shared_with_the_projections():
    """One buffer for attention whose keys are cut (few rows, a prompt), tq_gemv
    and tq_gemm in turn, eager and from a graph: the bits of calls with
    workspaces of their own."""
    import ternary_weight_base_amd as tq
    say("one workspace for attention and projections")
    rng = np.random.default_rng(900)
    sets = [_inputs(rng, 16, 2, 128, [(1, 5000), (2, 3000)]), _inputs(rng, 32, 8, 128, [(300, 5000)])]
    most = [5000, 5000]
    want = [_run(d, max_kv=m) for d, m in zip(sets, most)]
    shape = {1: (640, 5120), 16: (640, 5120), 100: (640, 5120)}
    blob = {m: upload_blob(B3, *weights(*nk, 40 + m)) for m, nk in shape.items()}
    acts = {m: (torch.randint(-127, 128, (m, nk[1]), dtype=torch.int8, device="cuda"), torch.rand(m, device="cuda")) for m, nk in shape.items()}
    need = [tq.tq_kv_attn_workspace_bytes(len(d["q"]), len(d["kv"]), d["q"].shape[1], d["ks"].shape[1], 128, m) for d, m in zip(sets, most)]
    proj = [tq.tq_gemv_workspace_bytes(B3, m, *shape[m]) for m in (1, 16)] + [tq.tq_gemm_workspace_bytes(B3, 100, *shape[100])]
    assert min(need) > 0 and max(proj) > 0, (need, proj)
    ws = torch.zeros(max(need + proj) // 4 + 4, dtype=torch.int32, device="cuda")
    y = {m: torch.empty((m, shape[m][0]), device="cuda") for m in shape}
    g = [{k: dev(v) for k, v in d.items()} for d in sets]
    outs = [torch.empty_like(x["q"]) for x in g]

    def product(m, w):
        (tq.tq_gemv if m <= 16 else tq.tq_gemm)(B3, m, *shape[m], blob[m], *acts[m], y[m], w)

    def attend(i):
        x = g[i]
        tq.tq_kv_attn(x["q"], x["cu"], x["kv"], x["table"], x["k"], x["v"], x["ks"], x["vs"], outs[i], most[i], ws=ws)

    def all_calls():
        for m, i in ((1, 0), (100, 1), (16, 0), (1, 1), (100, 0)):
            product(m, ws)
            attend(i)

    plain = {}
    for m in shape:
        own = torch.zeros(max(proj) // 4 + 4, dtype=torch.int32, device="cuda")
        product(m, own)
        plain[m] = y[m].clone()

    def check():
        torch.cuda.synchronize()
        assert int(torch.count_nonzero(ws)) == 0
        for m in shape:
            assert torch.equal(y[m], plain[m]), m
        for o, w in zip(outs, want):
            assert np.array_equal(o.cpu().numpy().view(np.uint16), w.view(np.uint16))
        for t in (*y.values(), *outs):
            t.fill_(float("nan"))

    all_calls()
    check()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            all_calls()
    for _ in range(3):
        torch.cuda.synchronize()
        graph.replay()
        check()


@pytest.mark.parametrize("rows,seqs,most", [(40, 40, 3000), (60, 12, 5000), (40, 40, 1000), (1040, 3, 20000), (700, 3, 20000)])
def test_graph_with_rows_dealt_anew(rows, seqs, most):
    """Captured once; then cu_rows and kv_len give the rows to other sequences:
    one row each, all rows to one sequence, rows of padding, sequences without
    any, contexts shorter and longer than they were."""
    import ternary_weight_base_amd as tq
    say(f"attention in a graph, {rows} rows of {seqs} sequences dealt anew")
    rng = np.random.default_rng(rows + seqs)
    hq, hkv, dim, longest = (16, 8, 64, most) if rows <= 60 else (4, 2, 128, 1500)
    d = _inputs(rng, hq, hkv, dim, [(rows // seqs + (s < rows % seqs), longest) for s in range(seqs)])
    g = {k: dev(v) for k, v in d.items()}
    out = torch.empty(d["q"].shape, dtype=torch.float16, device="cuda")
    ws = tq.kv_attn_workspace(rows, seqs, hq, hkv, dim, most)

    def call():
        tq.tq_kv_attn(g["q"], g["cu"], g["kv"], g["table"], g["k"], g["v"], g["ks"], g["vs"], out, most, ws=ws)

    call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    even = d["cu"].copy()
    first, last = np.full(seqs + 1, rows), np.zeros(seqs + 1)
    first[0] = 0
    last[-1] = rows
    some = np.minimum(np.arange(seqs + 1) // 2 * 2, rows - 5)  # every other one without rows, padding behind
    for cu in (even, first, last, some, np.sort(np.concatenate(([0], rng.integers(0, rows + 1, seqs - 1), [rows]))), even):
        d["cu"] = cu.astype(np.int32)
        d["kv"] = np.minimum(rng.integers(0, longest + 1, seqs) + np.diff(d["cu"]) // 2, longest).astype(np.int32)
        g["cu"].copy_(dev(d["cu"]))
        g["kv"].copy_(dev(d["kv"]))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        _check(d, got)
        assert np.array_equal(got.view(np.uint16), _run(d, max_kv=most).view(np.uint16))
        assert ws is None or int(torch.count_nonzero(ws)) == 0


def test_calls_on_two_streams_at_once():
    """Calls with workspaces of their own beside each other on two streams."""
    import ternary_weight_base_amd as tq
    say("attention on two streams at once")
    rng = np.random.default_rng(950)
    sets = [_inputs(rng, 16, 2, 128, [(1, 9000), (3, 4000)]), _inputs(rng, 32, 8, 128, [(300, 5000)])]
    want = [_run(d, max_kv=9000) for d in sets]
    g = [{k: dev(v) for k, v in d.items()} for d in sets]
    outs = [[torch.empty_like(x["q"]) for _ in range(20)] for x in g]
    spaces = [tq.kv_attn_workspace(len(d["q"]), len(d["kv"]), d["q"].shape[1], d["ks"].shape[1], 128, 9000) for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for n in range(20):
        for x, o, w, s in zip(g, outs, spaces, streams):
            tq.tq_kv_attn(x["q"], x["cu"], x["kv"], x["table"], x["k"], x["v"], x["ks"], x["vs"], o[n], 9000, ws=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert np.array_equal(x.cpu().numpy().view(np.uint16), w.view(np.uint16))
    assert all(int(torch.count_nonzero(w)) == 0 for w in spaces)
