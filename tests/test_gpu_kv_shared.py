"""tq_kv_attn_shared against the 64-bit attention over each sequence's whole
context: groups, prefixes and own parts of many sizes, every kernel for both
launches, and what the arrays may hold."""
import math

import numpy as np
import pytest

from gpu_util import dev, say
from kv_util import PAGE, attention, attention_tolerance

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(heads, groups, seed, alone=(), pad=0, flat_scales=False):
    """groups: [(prefix, [(rows, own tokens)...])...]; alone: sequences behind the last group."""
    hq, hkv, dim = heads
    rng = np.random.default_rng(seed)
    seqs, prefix, cu_seqs = [], [], [0]
    for p, members in groups:
        seqs += [(p, n, t) for n, t in members]
        prefix.append(p)
        cu_seqs.append(len(seqs))
    seqs += [(0, n, t) for n, t in alone]
    group_of = [g for g, (_, m) in enumerate(groups) for _ in m] + [-1] * len(alone)
    total = [p + t for p, n, t in seqs]
    shared = [p // PAGE for p in prefix]
    used = [max(0, math.ceil(t / PAGE)) - (shared[g] if g >= 0 else 0) for t, g in zip(total, group_of)]
    pages = sum(shared) + sum(max(u, 0) for u in used) + 3
    order, at = rng.permutation(pages), sum(shared)
    first = np.cumsum([0] + shared)
    width = max(math.ceil(t / PAGE) for t in total + [1]) + 2
    table = np.full((len(seqs), width), -1, np.int32)
    for s, (u, g) in enumerate(zip(used, group_of)):
        b = shared[g] if g >= 0 else 0
        if g >= 0:
            table[s, :b] = order[first[g]:first[g] + b]
        if u > 0:
            table[s, b:b + u] = order[at:at + u]
            at += u
    cu = np.cumsum([0] + [n for _, n, _ in seqs]).astype(np.int32)
    c = {"heads": heads, "q": (2 * rng.standard_normal((cu[-1] + pad, hq, dim))).astype(np.float16), "cu": cu,
         "kv": np.array(total, np.int32), "cu_seqs": np.array(cu_seqs, np.int32), "prefix": np.array(prefix, np.int32), "table": table,
         "k": rng.integers(0, 256, (pages, hkv, PAGE, dim), dtype=np.uint8), "v": rng.integers(0, 256, (pages, hkv, dim, PAGE), dtype=np.uint8)}
    e = (lambda: np.full((pages, hkv), -7)) if flat_scales else (lambda: rng.integers(-9, -4, (pages, hkv)))
    c["ks"], c["vs"] = (2.0 ** e()).astype(np.float32), (2.0 ** e()).astype(np.float32)
    c["most_prefix"] = max(prefix)
    c["most_own"] = max([t for _, _, t in seqs] + [1])
    return c


def call(c, ws=None, **more):
    import ternary_weight_base_amd as tq
    hq, hkv, dim = c["heads"]
    a = {n: dev(c[n]) for n in ("q", "cu", "kv", "cu_seqs", "prefix", "table", "k", "v", "ks", "vs")}
    a.update(more)
    out = more.get("out", torch.full(c["q"].shape, math.nan, dtype=torch.float16, device="cuda"))
    if ws is None:
        ws = tq.kv_attn_shared_workspace(c["q"].shape[0], len(c["kv"]), len(c["prefix"]), hq, hkv, dim, c["most_prefix"], c["most_own"])
    tq.tq_kv_attn_shared(a["q"], a["cu"], a["kv"], a["cu_seqs"], a["prefix"], a["table"], a["k"], a["v"], a["ks"], a["vs"], out,
                         c["most_prefix"], c["most_own"], ws=ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert int(ws.count_nonzero()) == 0, "the workspace must be left zero"
    return out


def verify(c, out):
    hq, hkv, dim = c["heads"]
    ref, mag, dot = attention(c["q"], c["cu"], c["kv"], c["table"], c["k"], c["v"], c["ks"], c["vs"], dim ** -0.5, 0, 0)
    # (the join's roundings: two weights, a product and a sum each, a quotient: within 8 more keys' worth)
    tol = attention_tolerance(ref, mag, dot, int(c["kv"].max()) + 8, dim)
    got = out.cpu().numpy().astype(np.float64)
    n = c["cu"][-1]
    assert np.isnan(got[n:]).all(), "rows behind the last sequence changed"
    err = np.abs(got[:n] - ref[:n])
    assert (err <= tol[:n]).all(), f"{np.nanmax(err / tol[:n])} of the tolerance"


def users(n, own, rows=1, seed=0):
    rng = np.random.default_rng(seed)
    return [(rows, int(max(rows, rng.integers(1, own + 1)))) for _ in range(n)]


def shares(c):
    """Whether the call takes two launches: its workspace is then not that of tq_kv_attn."""
    import ternary_weight_base_amd as tq
    n, (hq, hkv, dim) = (c["q"].shape[0], len(c["kv"])), c["heads"]
    return tq.tq_kv_attn_shared_workspace_bytes(*n, len(c["prefix"]), hq, hkv, dim, c["most_prefix"], c["most_own"]) != \
        tq.tq_kv_attn_workspace_bytes(*n, hq, hkv, dim, c["most_prefix"] + c["most_own"])


# What the call is told of its largest prefix and own part sets the kernels: larger
# numbers than there are take small inputs through all of them.  {name: (heads,
# groups, [(max_prefix_len, max_own_len; 0: as it is)...] that take two launches)}
LONG = 1 << 17
CASES = {
    "one_user": ((8, 2, 128), [(640, [(1, 30)])], []),
    # the prefix in tiles of 16 rows, cut; own parts whole, cut, in shares
    "two_users": ((16, 8, 128), [(2000, users(2, 90))], [(LONG, 0), (LONG, 30000)]),
    "two_users_64": ((16, 8, 64), [(9000, users(2, 200))], [(LONG, 0), (LONG, 30000)]),
    # ... in tiles of 32 rows
    "five_users": ((16, 4, 128), [(900, users(5, 300))], [(LONG, 0), (LONG, 30000)]),
    "five_users_64": ((16, 4, 64), [(5000, users(5, 1500, rows=2))], [(LONG, 0), (LONG, 30000)]),
    # ... whole, for many groups of few users
    "many_groups": ((8, 8, 64), [(64 * (i % 6), users(5, 40, seed=i)) for i in range(60)], [(1024, 0)]),
    "many_groups_128": ((32, 8, 128), [(64 * (i % 4) + 9, users(6, 30, seed=i)) for i in range(40)], [(1024, 0)]),
    "many_groups_16": ((16, 8, 128), [(64 * (i % 5), users(6, 30, seed=i)) for i in range(40)], [(1024, 0)]),
    # ... in tiles of 128 rows, in 32 pieces, fewer, one
    "many": ((64, 8, 128), [(2048, users(40, 200))], [(LONG, 0), (8192, 0)]),
    "many_64": ((16, 4, 64), [(1024, users(130, 70))], [(LONG, 0), (8192, 3000)]),
    "many_heads": ((64, 64, 64), [(300, users(150, 20))], [(320, 0), (4096, 0)]),
    "many_rows": ((16, 2, 64), [(700, users(30, 60, rows=5))], [(LONG, 0), (LONG, 30000)]),
    "many_long": ((32, 2, 128), [(6000, users(40, 300))], [(LONG, 0), (LONG, 30000)]),
    # own parts of thousands of tokens, several rows
    "long_own": ((8, 8, 64), [(128, users(30, 4000))], [(LONG, 0)]),
    "long_own_rows": ((16, 4, 128), [(192, users(12, 3000, rows=4))], [(LONG, 0), (LONG, 900)]),
    # own parts by the kernel for many rows: whole, cut
    "questions": ((16, 2, 64), [(512, [(8, 20), (7, 300), (5, 121), (6, 60)] * 16)], [(LONG, 0), (LONG, 3000)]),
    "questions_128": ((16, 2, 128), [(640, [(9, 900), (8, 31), (10, 1500)] * 8)], [(LONG, 0)]),
    "questions_few": ((8, 2, 64), [(512, [(70, 120), (60, 300), (50, 121), (60, 60)])], [(LONG, 0), (LONG, 2000)]),
    # groups of all sizes; prefixes of no page, of a part of one, of pages and a part
    "groups": ((8, 2, 128), [(0, users(3, 80)), (63, users(1, 5)), (64, users(4, 200)), (1000, users(20, 90)), (65, [(1, 1), (1, 64), (1, 63)])],
               [(LONG, 0), (LONG, 3000)]),
    "groups_rows": ((24, 4, 64), [(300, users(9, 300, rows=3)), (4100, users(2, 20, rows=2)), (128, [(0, 5), (7, 9), (0, 0)])],
                    [(LONG, 0), (LONG, 30000)]),
    "empty_groups": ((8, 4, 64), [(128, []), (640, users(3, 40)), (64, []), (256, users(1, 10)), (512, [])], []),
    "empty_groups_more": ((8, 4, 64), [(128, []), (640, users(13, 40)), (64, []), (256, users(4, 10)), (512, [])], [(LONG, 0), (LONG, 30000)]),
}


@pytest.mark.parametrize("name", CASES)
def test_cases(name):
    heads, groups, told = CASES[name]
    c = make(heads, groups, seed=len(name))
    most = c["most_prefix"], c["most_own"]
    for p, o in [(0, 0)] + told:
        c["most_prefix"], c["most_own"] = p or most[0], o or most[1]
        say(f"shared {name} {c['most_prefix']} {c['most_own']}")
        assert shares(c) or not p
        verify(c, call(c))


@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64), (6, 6, 64), (64, 8, 128), (33, 3, 128)], ids=str)
def test_sequences_outside_the_groups_and_padding(heads):
    c = make(heads, [(320, users(4, 100)), (128, users(2, 60))], seed=3, alone=[(1, 77), (0, 0), (3, 500), (1, 1)], pad=4)
    c["most_prefix"] = 1 << 22
    assert shares(c)
    verify(c, call(c))


@pytest.mark.parametrize("prefix", [0, 64, 1000])
def test_lengths_larger_than_there_are(prefix):
    """max_prefix_len and max_own_len only set the kernels."""
    for most_prefix, most_own in ((prefix, 130), (LONG, 130), (max(prefix, 64), 50000), (LONG, 20000)):
        c = make((8, 2, 64), [(prefix, users(6, 130))], seed=4)
        c["most_prefix"], c["most_own"] = most_prefix, most_own
        verify(c, call(c))


def test_strided_rows():
    c = make((6, 2, 64), [(200, users(5, 100, rows=2))], seed=5)
    c["most_prefix"] = LONG
    rows = c["q"].shape[0]
    wide = torch.full((rows, 6 * 64 + 40), math.nan, dtype=torch.float16, device="cuda")
    wide[:, :384] = dev(c["q"]).view(rows, 384)
    room = torch.full((rows, 6 * 64 + 8), math.nan, dtype=torch.float16, device="cuda")
    out = call(c, q=wide[:, :384].unflatten(1, (6, 64)), out=room[:, :384].unflatten(1, (6, 64)))
    verify(c, out)
    assert bool(torch.isnan(room[:, 384:]).all())


def test_in_place():
    """out may be q: own parts whole, cut, and rows of a prompt."""
    for heads, groups, told in (((8, 2, 64), [(200, users(5, 100, rows=2))], 0), ((16, 8, 128), [(2000, users(2, 90))], 30000),
                                ((16, 2, 64), [(512, [(8, 20), (7, 300), (5, 121), (6, 60)] * 4)], 3000)):
        c = make(heads, groups, seed=12)
        c["most_own"] = max(told, c["most_own"])
        for c["most_prefix"] in (LONG, 1 << 22):  # in one launch or two, in two
            assert shares(c) or c["most_prefix"] == LONG
            q = dev(c["q"])
            verify(c, call(c, q=q, out=q))


def test_missing_pages_and_scales_of_any_kind():
    """Pages outside the cache are not seen, in the prefix and behind it; pages of zeros."""
    c = make((8, 2, 128), [(640, users(9, 300)), (128, users(2, 70))], seed=6)
    n = c["ks"].shape[0]
    c["table"][:9, 3] = -1          # of the first prefix: the same for the group
    c["table"][:9, 7] = n + 5
    c["table"][4, 10] = -7          # of one sequence's own
    c["ks"][c["table"][0, 1]] = 0
    c["vs"][c["table"][0, 2]] = 0
    c["vs"][c["table"][9, 0]] = 0
    for c["most_prefix"] in (640, LONG):
        verify(c, call(c))


def test_rows_that_see_nothing():
    """A prefix and own pages that are all missing: zeros."""
    c = make((4, 2, 64), [(128, users(3, 40))], seed=7)
    c["table"][:] = -1
    for c["most_prefix"] in (128, LONG):
        assert not bool(call(c).any())


def test_large_scores_on_one_side():
    """All weight in the prefix, or none of it: scores hundreds apart."""
    for where in (0, 1):
        c = make((8, 2, 128), [(512, users(20, 100))], seed=8 + where, flat_scales=True)
        pages = c["table"][0, :8] if where == 0 else np.setdiff1d(np.arange(c["ks"].shape[0]), c["table"][0, :8])
        c["ks"][pages] *= 256
        c["most_prefix"] = LONG
        verify(c, call(c))


def test_the_same_as_without_sharing():
    """Against tq_kv_attn on the same arrays: two results of the same rows within both tolerances."""
    import ternary_weight_base_amd as tq
    c = make((16, 4, 128), [(1500, users(17, 400)), (300, users(5, 80, rows=2))], seed=10)
    most = int(c["kv"].max())
    c["most_prefix"] = LONG
    out = call(c)
    a = {n: dev(c[n]) for n in ("q", "cu", "kv", "table", "k", "v", "ks", "vs")}
    plain = torch.empty_like(a["q"])
    ws = tq.kv_attn_workspace(c["q"].shape[0], len(c["kv"]), 16, 4, 128, most)
    tq.tq_kv_attn(a["q"], a["cu"], a["kv"], a["table"], a["k"], a["v"], a["ks"], a["vs"], plain, most, ws=ws)
    verify(c, plain)
    verify(c, out)


def test_bad_arrays_stay_inside():
    for cu_seqs, prefix, cu in (([0, 9, 3, 40], [640, 1 << 30, -5], None), ([5, 2, -3, 1 << 30], [64, 128, 640], None),
                                ([0, 2, 4, 6], [640, 640, 640], [0, 5, 3, 99, -7, 2, 6])):
        c = make((8, 2, 64), [(640, users(2, 50)) for _ in range(3)], seed=11)
        c["cu_seqs"], c["prefix"] = np.array(cu_seqs, np.int32), np.array(prefix, np.int32)
        if cu is not None:
            c["cu"] = np.array(cu, np.int32)
        import ternary_weight_base_amd as tq
        ws = tq.kv_attn_shared_workspace(6, 6, 3, 8, 2, 64, LONG, 50)
        a = {n: dev(c[n]) for n in ("q", "cu", "kv", "cu_seqs", "prefix", "table", "k", "v", "ks", "vs")}
        out = torch.empty_like(a["q"])
        tq.tq_kv_attn_shared(a["q"], a["cu"], a["kv"], a["cu_seqs"], a["prefix"], a["table"], a["k"], a["v"], a["ks"], a["vs"], out, LONG, 50, ws=ws)
        torch.cuda.synchronize()


def test_captured_with_changing_groups():
    """One graph, replayed with other lengths, groups and rows; other calls on the same workspace between."""
    import ternary_weight_base_amd as tq
    heads = (16, 4, 64)
    cases = [make(heads, g, seed=20 + i) for i, g in enumerate((
        [(640, users(6, 300)), (2000, users(6, 900, seed=1))], [(64, users(1, 30)), (1900, users(11, 800, seed=2))],
        [(0, users(9, 900, seed=3)), (1000, [(1, 5), (0, 3), (1, 900)])], [(1280, users(10, 40)), (128, users(2, 1))]))]
    pages, width = max(c["ks"].shape[0] for c in cases), max(c["table"].shape[1] for c in cases)
    for c in cases:
        more = pages - c["ks"].shape[0]
        c["table"] = np.pad(c["table"], ((0, 0), (0, width - c["table"].shape[1])), constant_values=-1)
        for n in ("k", "v", "ks", "vs"):
            c[n] = np.pad(c[n], ((0, more),) + ((0, 0),) * (c[n].ndim - 1))
        c["q"] = np.pad(c["q"], ((0, 12 - c["q"].shape[0]), (0, 0), (0, 0)))
        c["most_prefix"], c["most_own"] = LONG, 900
        assert shares(c)
    ws = tq.kv_attn_shared_workspace(12, 12, 2, *heads, LONG, 900)
    a = {n: dev(cases[0][n]) for n in ("q", "cu", "kv", "cu_seqs", "prefix", "table", "k", "v", "ks", "vs")}
    out = torch.empty_like(a["q"])
    run = lambda: tq.tq_kv_attn_shared(a["q"], a["cu"], a["kv"], a["cu_seqs"], a["prefix"], a["table"], a["k"], a["v"], a["ks"], a["vs"],
                                       out, LONG, 900, ws=ws)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for c in cases + cases[::-1]:
        for n in a:
            a[n].copy_(dev(c[n]))
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert int(ws.count_nonzero()) == 0
        verify(c, out)
        assert torch.equal(call(c, ws=ws)[:c["cu"][-1]], out[:c["cu"][-1]])
