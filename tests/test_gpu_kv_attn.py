"""tq_kv_attn against a plain 64-bit attention over the values that the
cache's bytes stand for."""
import numpy as np
import pytest

from gpu_util import dev, say
from kv_util import PAGE, attention, attention_tolerance, lay_out

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(rng, hq, hkv, dim, lens, pad=0, spread=1.0, unused=-1):
    kv_len = np.array([t for _, t in lens], np.int32)
    cu = np.cumsum([0] + [n for n, _ in lens]).astype(np.int32)
    table, pages = lay_out(rng, kv_len, unused=unused)
    d = {"q": (spread * rng.standard_normal((cu[-1] + pad, hq, dim))).astype(np.float16), "cu": cu, "kv": kv_len, "table": table,
         "k": rng.integers(0, 256, (pages, hkv, PAGE, dim), dtype=np.uint8),
         "v": rng.integers(0, 256, (pages, hkv, dim, PAGE), dtype=np.uint8),
         "ks": (2.0 ** rng.integers(-8, -4, (pages, hkv))).astype(np.float32),
         "vs": (2.0 ** rng.integers(-8, -4, (pages, hkv))).astype(np.float32)}
    return d


def _run(d, window=0, sinks=0, scale=None, max_kv=None, ws=None, out=None):
    import ternary_weight_base_amd as tq
    rows, hq, dim = d["q"].shape
    g = {k: dev(v) for k, v in d.items()}
    if out is None:
        out = torch.full((rows, hq, dim), float("nan"), dtype=torch.float16, device="cuda")
    # (a large max_kv_len: the kernel for many rows takes these sizes already)
    most = max_kv or (20000 if rows > 1000 else max(1, int(d["kv"].max())))
    if ws is None:
        ws = tq.kv_attn_workspace(rows, len(d["kv"]), hq, d["ks"].shape[1], dim, most)
    tq.tq_kv_attn(g["q"], g["cu"], g["kv"], g["table"], g["k"], g["v"], g["ks"], g["vs"], out, most, softmax_scale=scale,
                  window=window, sinks=sinks, ws=ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert int(torch.count_nonzero(ws)) == 0, "workspace left non-zero"
    return out.cpu().numpy()


def _check(d, got, window=0, sinks=0, scale=None):
    dim = d["q"].shape[2]
    ref, mag, dot = attention(d["q"], d["cu"], d["kv"], d["table"], d["k"], d["v"], d["ks"], d["vs"],
                              dim ** -0.5 if scale is None else scale, window, sinks)
    pad = np.isnan(ref)
    assert np.all(np.isnan(got[pad])), "rows behind the last sequence were written"
    tol = attention_tolerance(ref, mag, dot, max(1, int(d["kv"].max())), dim)
    err = np.abs(got.astype(np.float64) - ref)
    bad = ~pad & ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}, tolerance {tol[bad][0]}"


CASES = [
    # (hq, hkv, dim, [(rows, kv_len)...], window, sinks, padding rows)
    (8, 1, 128, [(1, 1)], 0, 0, 0),
    (8, 2, 128, [(1, 63), (1, 64), (1, 65), (1, 2)], 0, 0, 1),
    (4, 4, 64, [(1, 500), (0, 100), (1, 1), (1, 1300)], 0, 0, 0),
    (5, 1, 128, [(3, 300), (1, 77), (0, 0), (7, 7)], 0, 0, 2),
    (6, 2, 64, [(17, 200), (2, 129)], 0, 0, 0),
    (24, 1, 64, [(2, 70)], 0, 0, 0),
    (12, 1, 128, [(1, 4097)], 0, 0, 0),
    (2, 1, 128, [(5, 3), (2, 0), (1, 1)], 0, 0, 0),          # rows before position 0 see nothing
    (8, 1, 128, [(1, 1000), (1, 70), (1, 5)], 100, 0, 0),
    (4, 2, 64, [(1, 1000), (3, 700), (1, 129)], 64, 4, 0),
    (4, 2, 64, [(40, 1000)], 1, 0, 0),                        # each row sees itself
    (8, 1, 128, [(33, 900), (70, 130)], 200, 70, 3),
    (8, 1, 64, [(1, 900)], 2000, 5, 0),                       # a window longer than the sequence
    (8, 2, 128, [(130, 130)], 0, 0, 0),
    (4, 4, 64, [(200, 413), (65, 65)], 0, 0, 5),
    (40, 8, 128, [(31, 700)], 0, 0, 0),
    (7, 1, 128, [(90, 290), (1, 2000), (0, 5), (12, 12)], 0, 0, 0),
    (16, 2, 128, [(300, 500)], 77, 130, 0),
    (2, 2, 128, [(1, 1 + 13 * i) for i in range(90)], 0, 0, 0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(i):
    hq, hkv, dim, lens, window, sinks, pad = CASES[i]
    say(f"attention case {i}: {CASES[i][:3]} {lens[:5]} window {window} sinks {sinks}")
    d = _inputs(np.random.default_rng(200 + i), hq, hkv, dim, lens, pad)
    _check(d, _run(d, window, sinks), window, sinks)


# as above, and max_kv_len: sizes that the kernel for many rows takes
MANY = [
    (8, 8, 128, [(520, 520)], 0, 0, 0, 20000),
    (16, 16, 64, [(1100, 1100)], 0, 0, 0, None),
    (8, 4, 64, [(700, 900), (0, 3), (333, 333)], 0, 0, 3, 20000),
    (16, 2, 128, [(300, 500)], 77, 130, 0, 20000),
    (40, 8, 128, [(131, 700)], 0, 0, 1, 20000),
    (7, 1, 128, [(700, 790), (90, 2000), (0, 5), (12, 12)], 0, 0, 2, 20000),
    (4, 2, 64, [(1400, 1000)], 1, 0, 0, 20000),             # rows before position 0, each row sees itself
    (8, 8, 64, [(530, 600), (530, 20)], 2000, 5, 0, 20000),
    (8, 8, 128, [(530, 900), (70, 130)], 200, 70, 3, 20000),
    (32, 8, 128, [(300, 9001)], 0, 0, 0, None),             # keys in pieces
    (24, 4, 64, [(260, 7000), (400, 4001)], 0, 0, 5, None),
    (32, 8, 128, [(300, 5000), (10, 70)], 3001, 64, 0, None),
    (4, 1, 128, [(4100, 4160)], 64, 4, 0, 20000),
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_many_rows(i):
    hq, hkv, dim, lens, window, sinks, pad, most = MANY[i]
    say(f"attention of many rows, case {i}: {MANY[i]}")
    d = _inputs(np.random.default_rng(300 + i), hq, hkv, dim, lens, pad)
    got = _run(d, window, sinks, max_kv=most)
    _check(d, got, window, sinks)
    assert np.array_equal(got.view(np.uint16), _run(d, window, sinks, max_kv=most).view(np.uint16))


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_split_keys(rows, dim):
    """A long context cut into many pieces; twice with the same result, bit for
    bit; a workspace for less than the length."""
    say(f"attention split, {rows} rows, dim {dim}")
    d = _inputs(np.random.default_rng(31), 8, 1, dim, [(rows, 9001), (rows, 130)])
    a = _run(d)
    _check(d, a)
    assert np.array_equal(a.view(np.uint16), _run(d).view(np.uint16))
    _check(d, _run(d, max_kv=1))
    _check(d, _run(d, max_kv=100000))


def test_decode_is_the_rounded_result():
    """One row a sequence: the rounding of the weights to fp16 is compensated,
    so nearly every output is the correctly rounded one.  A score is about
    2 * 128 + 16 roundings of 2^-24 of sum |q||k| scale (below 2^4 here) away
    from exact, in the root-sum 2^4.05 * 2^-24 * 2^4 = 2^-16 of a weight at most; independent over the keys, so as much
    of the output, whose rounding borders lie 2^-11 apart at least: at most 2 * 2^-16 / 2^-11 = 1 in 16
    outputs next to one.  (Weights rounded to 2^-11, rms 2^-12.3, would change one in four.)"""
    say("attention decode precision")
    d = _inputs(np.random.default_rng(41), 8, 1, 128, [(1, 2000)], spread=0.6)
    got = _run(d)
    ref, _, dot = attention(d["q"], d["cu"], d["kv"], d["table"], d["k"], d["v"], d["ks"], d["vs"], 128 ** -0.5, 0, 0)
    assert dot.max() < 16
    assert np.mean(got != ref.astype(np.float16)) <= 1 / 16


def test_scales_apart_and_zero_pages():
    """Value scales of neighbouring pages far apart, pages of zeros (scale 0), any positive scale."""
    say("attention scales")
    rng = np.random.default_rng(51)
    for lens in ([(1, 600), (2, 64)], [(60, 640)], [(1040, 1100)]):
        d = _inputs(rng, 4, 2, 128, lens)
        n = d["vs"].shape[0]
        d["vs"] = (2.0 ** rng.integers(-24, 4, d["vs"].shape)).astype(np.float32)
        d["vs"][rng.permutation(n)[:n // 3]] = 0
        d["ks"][rng.permutation(n)[:n // 4]] = 0
        _check(d, _run(d))
        d["ks"] = rng.uniform(1e-3, 2e-2, d["ks"].shape).astype(np.float32)
        d["vs"] = np.exp(rng.uniform(-9, 2, d["vs"].shape)).astype(np.float32)
        _check(d, _run(d))


def test_value_scales_from_one_end_to_the_other():
    """Pages whose values are below all that fp16 holds, before, behind and
    between pages of large ones (dropped, they are worth less than 2^-33)."""
    say("attention value scales 2^-126 .. 2^8")
    rng = np.random.default_rng(53)
    for lens in ([(1, 900)], [(1, 9000)], [(5, 1500)], [(60, 900)], [(1100, 1200)]):
        d = _inputs(rng, 4, 1, 128, lens)
        ids = d["table"][0, :-(-lens[0][1] // PAGE)]
        place = np.arange(len(ids))
        for small in (place * 2 >= len(ids), place * 2 < len(ids), place % 16 < 8, place % 2 == 0, place >= 0):
            for tiny in (2.0 ** -110, 2.0 ** -126):
                d["vs"][ids, 0] = np.where(small, tiny, 2.0 ** 8)
                _check(d, _run(d))


def test_unused_places_do_not_matter():
    """NaN and infinite scales in pages that no sequence holds, and other
    bytes behind the last token: the same output bits."""
    say("attention garbage")
    rng = np.random.default_rng(61)
    for lens in ([(1, 70), (1, 1)], [(50, 100)], [(1040, 1100)]):
        d = _inputs(rng, 4, 1, 64, lens)
        a = _run(d)
        held = set()
        for s, (_, t) in enumerate(lens):
            ids = d["table"][s, :-(-t // PAGE)]
            held |= set(ids.tolist())
            if t % PAGE:
                d["k"][ids[-1], :, t % PAGE:] = 255
                d["v"][ids[-1], :, :, t % PAGE:] = 0
        for p in range(len(d["ks"])):
            if p not in held:
                d["ks"][p], d["vs"][p] = np.nan, np.inf
        d["table"][d["table"] == -1] = 1 << 30
        assert np.array_equal(a.view(np.uint16), _run(d).view(np.uint16))
        _check(d, a)


def test_holes_and_lengths_beyond_the_table():
    say("attention holes")
    rng = np.random.default_rng(71)
    for lens in ([(1, 400), (2, 300), (1, 64)], [(70, 400), (33, 290), (1, 1)], [(1040, 1200), (300, 400), (1, 1)]):
        d = _inputs(rng, 4, 2, 128, lens)
        d["table"][0, 1], d["table"][0, 4], d["table"][1, 0] = -1, 1 << 20, -9
        d["table"][2, 0] = len(d["ks"])  # all that this sequence has
        _check(d, _run(d))
        d["kv"][0] = 64 * d["table"].shape[1] + 30  # rows behind the page table see what there is
        _check(d, _run(d))
        _check(d, _run(d, 100, 3), 100, 3)


def test_rows_out_of_order_touch_nothing_else():
    """cu_rows that is not ascending, or points outside: whatever the rows get,
    the workspace is left zero and a following call is right."""
    import ternary_weight_base_amd as tq
    say("attention with bad cu_rows")
    rng = np.random.default_rng(75)
    for lens in ([(1, 2000), (2, 300), (1, 64)], [(70, 400), (33, 290), (1, 1)], [(1, 90)] * 3, [(1000, 1100), (33, 290), (1, 1)]):
        d = _inputs(rng, 4, 2, 128, lens)
        rows = d["q"].shape[0]
        ws = torch.zeros(tq.tq_kv_attn_workspace_bytes(rows, 3, 4, 2, 128, 20000 if rows > 1000 else int(d["kv"].max())) // 4 + 4, dtype=torch.int32, device="cuda")
        good = _run(d, ws=ws)
        for cu in ([0, rows, 0, rows], [5, -3, rows + 9, 1 << 30], [rows, 1, 1, 0], [-1 << 30, rows, rows, rows], [1, 1, 1, 1]):
            _run({**d, "cu": np.array(cu, np.int32)}, ws=ws)
        assert np.array_equal(_run(d, ws=ws).view(np.uint16), good.view(np.uint16))


def test_largest_window_and_rows_before_the_start():
    """A window and sinks as large as their type holds, with rows at negative positions."""
    say("attention largest window")
    rng = np.random.default_rng(76)
    for lens in ([(80, 60), (3, 2)], [(3, 2), (1, 40)], [(200, 190)], [(1100, 1070)]):
        d = _inputs(rng, 4, 1, 64, lens)
        for window, sinks in ((0x7fffffff, 0), (0x7fffffff, 0x7fffff00), (0x7ffffff0, 1)):
            _check(d, _run(d, window, sinks), window, sinks)


def test_cache_beyond_32_bits():
    """Pages whose bytes lie past 4 GiB in each cache, appended to and read."""
    import ternary_weight_base_amd as tq
    say("cache of more than 4 GiB")
    rng = np.random.default_rng(77)
    pages, hkv, dim, hq = 66000, 8, 128, 8
    k, v = (torch.empty((pages, hkv) + s, dtype=torch.uint8, device="cuda") for s in ((PAGE, dim), (dim, PAGE)))
    assert k.numel() > 1 << 32
    ks, vs = torch.empty((pages, hkv), device="cuda"), torch.empty((pages, hkv), device="cuda")
    for n in (1, 150):
        used = pages - 1 - rng.permutation(400)[:3]
        lens = np.array([n], np.int32)
        table = np.full((1, 3), -1, np.int32)
        table[0, :-(-n // PAGE)] = used[:-(-n // PAGE)]
        x = rng.standard_normal((n, (hq + 2 * hkv) * dim)).astype(np.float32)
        q, out = (torch.empty((n, hq, dim), dtype=torch.float16, device="cuda") for _ in range(2))
        cu = dev(np.array([0, n], np.int32))
        tq.tq_kv_append(dev(x), None, cu, dev(lens), dev(table), k, v, ks, vs, q)
        tq.tq_kv_attn(q, cu, dev(lens), dev(table), k, v, ks, vs, out, n, ws=tq.kv_attn_workspace(n, 1, hq, hkv, dim, n))
        ids = torch.from_numpy(used.astype(np.int64)).cuda()
        small = np.array([[0, 1, 2]], np.int32)
        d = {"q": q.cpu().numpy(), "cu": np.array([0, n]), "kv": lens, "table": small, "k": k[ids].cpu().numpy(), "v": v[ids].cpu().numpy(),
             "ks": ks[ids].cpu().numpy(), "vs": vs[ids].cpu().numpy()}
        assert np.array_equal(d["q"], x[:, :hq * dim].reshape(n, hq, dim).astype(np.float16))
        for name, xs, c, s in (("k", x[:, hq * dim:(hq + hkv) * dim], d["k"], d["ks"]), ("v", x[:, (hq + hkv) * dim:], d["v"].transpose(0, 1, 3, 2), d["vs"])):
            got = ((c.astype(np.float64) - 127.5) * s[:, :, None, None]).transpose(0, 2, 1, 3).reshape(3 * PAGE, hkv, dim)[:n]
            half = np.repeat(s, PAGE, 0)[:n, :, None] / 2
            assert np.all(np.abs(got - xs.reshape(n, hkv, dim)) <= half), name
        _check(d, out.cpu().numpy())
    del k, v
    torch.cuda.empty_cache()


def test_sharp_scores_and_large_queries():
    """A softmax that picks one key, and scores that grow along the keys (the
    running maximum moves in every tile)."""
    say("attention sharp")
    rng = np.random.default_rng(81)
    for lens in ([(1, 900)], [(64, 900)], [(1040, 1100)]):
        d = _inputs(rng, 4, 1, 128, lens, spread=30.0)
        _check(d, _run(d))
        d["q"][:] = np.abs(d["q"]) / 8
        d["k"][:] = 0
        t = lens[0][1]
        for j in range(t):
            d["k"][d["table"][0, j // PAGE], :, j % PAGE] = min(255, j // 4)
        d["ks"][:] = 2.0 ** -7
        _check(d, _run(d))


def test_infinite_and_nan_queries_stay_in_their_row():
    say("attention nan")
    rng = np.random.default_rng(91)
    for lens in ([(2, 200), (1, 90)], [(80, 200)], [(1040, 1100)]):
        d = _inputs(rng, 4, 2, 64, lens)
        clean = _run(d)
        d["q"][1, 2, 5] = np.nan
        got = _run(d)
        assert np.all(np.isnan(got[1, 2]))
        got[1, 2] = clean[1, 2]
        assert np.array_equal(got.view(np.uint16), clean.view(np.uint16))


def test_strided_and_in_place():
    import ternary_weight_base_amd as tq
    say("attention strides")
    rng = np.random.default_rng(95)
    for lens in ([(1, 300), (1, 50)], [(50, 300)], [(1040, 1100)]):
        d = _inputs(rng, 4, 2, 128, lens)
        want = _run(d)
        rows = d["q"].shape[0]
        wide = torch.full((rows, 4 * 128 + 64), float("nan"), dtype=torch.float16, device="cuda")
        qs = wide[:, 32:32 + 512].unflatten(1, (4, 128))
        qs.copy_(dev(d["q"]))
        g = {k: dev(v) for k, v in d.items()}
        most = 20000 if rows > 1000 else 300
        ws = tq.kv_attn_workspace(rows, len(d["kv"]), 4, 2, 128, most)
        tq.tq_kv_attn(qs, g["cu"], g["kv"], g["table"], g["k"], g["v"], g["ks"], g["vs"], qs, most, ws=ws)
        assert np.array_equal(qs.cpu().numpy().view(np.uint16), want.view(np.uint16))
        assert torch.isnan(wide[:, :32]).all() and torch.isnan(wide[:, 544:]).all()


def test_side_stream_and_shared_workspace():
    """Another stream than the tensors'; one workspace for calls of several shapes in turn, and for tq_gemv."""
    import ternary_weight_base_amd as tq
    say("attention side stream")
    rng = np.random.default_rng(97)
    a, b = _inputs(rng, 8, 1, 128, [(1, 5000)]), _inputs(rng, 4, 4, 64, [(2, 3001), (1, 700)])
    wa, wb = _run(a), _run(b)
    need = max(tq.tq_kv_attn_workspace_bytes(1, 1, 8, 1, 128, 5000), tq.tq_kv_attn_workspace_bytes(3, 2, 4, 4, 64, 3001))
    ws = torch.zeros(need // 4 + 8, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            assert np.array_equal(_run(a, ws=ws).view(np.uint16), wa.view(np.uint16))
            assert np.array_equal(_run(b, ws=ws).view(np.uint16), wb.view(np.uint16))


def test_graph_replay_with_new_lengths():
    """Captured once at the longest length; the lengths change between replays."""
    import ternary_weight_base_amd as tq
    say("attention in a graph")
    rng = np.random.default_rng(99)
    d = _inputs(rng, 8, 2, 128, [(1, 3000), (1, 2000), (1, 900)])
    g = {k: dev(v) for k, v in d.items()}
    out = torch.empty((3, 8, 128), dtype=torch.float16, device="cuda")
    ws = tq.kv_attn_workspace(3, 3, 8, 2, 128, 3000)

    def call():
        tq.tq_kv_attn(g["q"], g["cu"], g["kv"], g["table"], g["k"], g["v"], g["ks"], g["vs"], out, 3000, ws=ws)

    call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    junk = torch.randn(1 << 18, device="cuda")
    for lens in ([3000, 2000, 900], [1, 64, 65], [0, 1999, 3], [2999, 1, 0], [3000, 2000, 900]):
        d["kv"][:] = lens
        g["kv"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        junk.mul_(1.0001)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        _check(d, got)
        assert np.array_equal(got.view(np.uint16), _run(d, max_kv=3000).view(np.uint16))
        assert int(torch.count_nonzero(ws)) == 0


def test_two_graphs_share_a_workspace():
    """A prompt's piece whose keys are cut, and one token over a long context,
    captured apart with one workspace, replayed in turn."""
    import ternary_weight_base_amd as tq
    say("attention, two graphs")
    rng = np.random.default_rng(103)
    sets = [_inputs(rng, 32, 8, 128, [(300, 5000)]), _inputs(rng, 16, 2, 128, [(1, 9000)]), _inputs(rng, 8, 1, 64, [(9, 4000)])]
    want = [_run(d) for d in sets]
    shapes = [(d["q"].shape[0], 1, d["q"].shape[1], d["ks"].shape[1], d["q"].shape[2], int(d["kv"][0])) for d in sets]
    need = [tq.tq_kv_attn_workspace_bytes(*s) for s in shapes]
    assert min(need) > 0
    ws = torch.zeros(max(need) // 4, dtype=torch.int32, device="cuda")
    g = [{k: dev(v) for k, v in d.items()} for d in sets]
    outs = [torch.empty(d["q"].shape, dtype=torch.float16, device="cuda") for d in sets]
    graphs = []
    s = torch.cuda.Stream()
    for x, out, shape in zip(g, outs, shapes):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                tq.tq_kv_attn(x["q"], x["cu"], x["kv"], x["table"], x["k"], x["v"], x["ks"], x["vs"], out, shape[5], ws=ws)
        graphs.append(graph)
    for order in ((0, 1, 2), (2, 0, 1, 1), (1, 2, 2, 0)):
        for i in order:
            outs[i].fill_(float("nan"))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert np.array_equal(outs[i].cpu().numpy().view(np.uint16), want[i].view(np.uint16)), i
        assert int(torch.count_nonzero(ws)) == 0


def test_long_prompt_against_its_own_last_rows():
    """12000 rows at once, and rows of it asked for alone: the kernels for many
    and for few rows, each within its distance from exact, agree."""
    import ternary_weight_base_amd as tq
    say("attention of 12000 rows")
    hq, hkv, dim, n, t = 16, 2, 128, 12000, 16000
    gen = torch.Generator(device="cuda").manual_seed(5)
    pages = t // PAGE
    q = torch.randn((n, hq, dim), generator=gen, device="cuda").half()
    k, v = (torch.randint(0, 256, (pages, hkv) + s, generator=gen, device="cuda", dtype=torch.uint8) for s in ((PAGE, dim), (dim, PAGE)))
    ks, vs = (torch.full((pages, hkv), 2.0 ** -6, device="cuda") for _ in range(2))
    table = torch.randperm(pages, generator=gen, device="cuda").int()[None]
    out = torch.empty_like(q)
    cu = dev(np.array([0, n], np.int32))

    def call(qq, o, cu, last):
        kv = dev(np.array([last], np.int32))
        tq.tq_kv_attn(qq, cu, kv, table, k, v, ks, vs, o, last, ws=tq.kv_attn_workspace(qq.shape[0], 1, hq, hkv, dim, last))

    call(q, out, cu, t)
    for first in (0, 1, 4000, 7777, n - 3):
        few = torch.empty((3, hq, dim), dtype=torch.float16, device="cuda")
        call(q[first:first + 3], few, dev(np.array([0, 3], np.int32)), t - n + first + 3)
        # weights off by 2^-11 and little else, values up to 2 (2^7 codes of 2^-6), two outputs rounded to fp16
        err = (out[first:first + 3].double() - few.double()).abs().max()
        assert float(err) <= 2 * 2 * 2.0 ** -11 + 2 * 2.0 ** -11, first
