"""tq_linear_attn against the recurrence in float64: both forms, head
layouts, lengths, decays, strides, states read and written, sizes of input."""
import math

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(heads, n, dtype, decay, seed, size=1.0, pad=0, extra=2):
    """Inputs of sequences of n rows: start and target states scattered over a pool."""
    hq, hkv, dim = heads
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, seqs = sum(n) + pad, len(n)
    qkv = (size * torch.randn((rows, (hq + 2 * hkv) * dim), generator=g, device="cuda")).to(dtype)
    if decay == "heads":
        d = -torch.exp2(torch.linspace(-10, 2, hkv, device="cuda"))
    else:
        d = -torch.rand((rows, hkv), generator=g, device="cuda") ** 4
    if decay == "odd":  # none, growth, resets, far below any fp32 factor
        d[torch.rand((rows, hkv), generator=g, device="cuda") < 0.3] = 0.0
        for v, p in ((0.5, 0.02), (-math.inf, 0.02), (-150.0, 0.02), (-1e30, 0.01)):
            d[torch.rand((rows, hkv), generator=g, device="cuda") < p] = v
    states = 2 * size * size * torch.randn((2 * seqs + extra, hkv, dim, dim), generator=g, device="cuda")
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    order = torch.randperm(2 * seqs, generator=g, device="cuda").int()
    return {"qkv": qkv, "decay": d, "states": states, "cu": cu, "from": order[:seqs].tolist(), "to": order[seqs:].tolist(), "heads": heads,
            "scale": 1.0 / math.sqrt(dim) / size ** 3}


def call(c, qkv=None, decay=None, out=None, states=None, scratch=None):
    import ternary_weight_base_amd as tq
    hq, hkv, dim = c["heads"]
    rows = c["qkv"].shape[0]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    states = c["states"].clone() if states is None else states
    if out is None:
        out = torch.full((rows, hq, dim), math.nan, dtype=torch.float16, device="cuda")
    if scratch is None:
        scratch = tq.linear_attn_scratch(rows, len(c["from"]), hq, hkv, dim)
        if scratch is not None:
            scratch.fill_(-1)  # NaN: nothing may rely on its contents
    tq.tq_linear_attn(c["qkv"] if qkv is None else qkv, c["decay"] if decay is None else decay, dev(c["cu"]), dev(c["from"]),
                      dev(c["to"]), states, out, scale=c["scale"], scratch=scratch)
    torch.cuda.synchronize()
    return out, states


def verify(c, out, states):
    from linear_util import check
    hq, hkv, dim = c["heads"]
    # check() reads the pool as it was before the call
    check(out, states, c["qkv"], c["decay"], c["cu"], c["from"], c["to"], c["states"], c["scale"], hq, hkv, dim)


HEADS = [(8, 1, 128), (4, 4, 64), (6, 2, 128), (5, 1, 64), (2, 2, 128), (33, 3, 64)]
LENGTHS = {"one": [1], "ones": [1] * 9, "few": [3, 0, 1, 9, 16], "seventeen": [17], "edges": [127, 128, 129, 1, 0, 64, 65, 33],
           "long": [700, 130]}


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_shapes(heads, lengths, dtype):
    say(f"linear {heads} {lengths} {dtype}")
    dt = {"f16": torch.float16, "f32": torch.float32}[dtype]
    c = make(heads, LENGTHS[lengths], dt, "heads" if heads[1] > 2 else "rows", seed=sum(heads) + len(lengths))
    verify(c, *call(c))


@pytest.mark.parametrize("n", [[5, 1, 3], [300, 140]], ids=["rows", "chunks"])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_decays_at_their_ends(n, dtype):
    dt = {"f16": torch.float16, "f32": torch.float32}[dtype]
    c = make((4, 2, 128), n, dt, "odd", seed=5)
    verify(c, *call(c))


@pytest.mark.parametrize("n", [[5, 1, 3], [150, 290]], ids=["rows", "chunks"])
@pytest.mark.parametrize("dtype,size", [("f16", 1e-4), ("f16", 2000.0), ("f32", 1e-9), ("f32", 1e9)])
def test_sizes_of_input(n, dtype, size):
    """fp16 keys up to their end, fp32 inputs far outside fp16's range (the scale brings the outputs back)."""
    dt = {"f16": torch.float16, "f32": torch.float32}[dtype]
    c = make((4, 2, 64), n, dt, "rows", seed=6, size=size)
    verify(c, *call(c))


def test_tokens_of_very_different_size():
    """A few rows thousands of times larger than the others, before and behind resets."""
    c = make((2, 1, 128), [400], torch.float32, "odd", seed=7)
    c["qkv"][::37] *= 5000.0
    verify(c, *call(c))


@pytest.mark.parametrize("n", [[4, 2, 7], [200, 3, 150]], ids=["rows", "chunks"])
def test_starts_and_targets(n):
    # from nothing, to nowhere, in place, two from the same start
    c = make((4, 2, 64), n, torch.float16, "rows", seed=8)
    a, b = c["from"], c["to"]
    num = c["states"].shape[0]
    for start, to in (([-1, a[1], num], b), (a, [-1, b[1], 1 << 30]), (a, a), ([a[0]] * 3, b), ([-5, -1, -1], [-1, -2, num])):
        c["from"], c["to"] = start, to
        verify(c, *call(c))


@pytest.mark.parametrize("n", [[4, 2, 7], [200, 3, 150]], ids=["rows", "chunks"])
def test_strided_rows_and_padding(n):
    c = make((6, 3, 64), n, torch.float32, "rows", seed=9, pad=5)
    rows, width = c["qkv"].shape
    wide = torch.full((rows, width + 24), math.nan, device="cuda")
    wide[:, :width] = c["qkv"]
    d = torch.full((rows, 7), math.nan, device="cuda")
    d[:, 2:5] = c["decay"]
    room = torch.full((rows, 6 * 64 + 40), math.nan, dtype=torch.float16, device="cuda")
    out = room[:, :384].unflatten(1, (6, 64))
    got, states = call(c, qkv=wide[:, :width], decay=d[:, 2:5], out=out)
    verify(c, got, states)
    assert bool(torch.isnan(room[:, 384:]).all())


@pytest.mark.parametrize("n", [[3, 2, 8], [129, 40]], ids=["rows", "chunks"])
def test_rows_far_apart(n):
    """Rows of qkv 2^25 elements apart and of out 2^22: byte offsets past 32 and up to 31 bits."""
    c = make((2, 1, 64), n, torch.float16, "rows", seed=19)
    rows = sum(n)
    qkv = torch.empty((rows, 1 << 25), dtype=torch.float16, device="cuda")[:, :4 * 64]
    qkv.copy_(c["qkv"])
    room = torch.full((rows, 1 << 22), math.nan, dtype=torch.float16, device="cuda")
    got, states = call(c, qkv=qkv, out=room[:, :128].unflatten(1, (2, 64)))
    verify(c, got, states)
    assert bool(torch.isnan(room[:, 128:]).all())


def test_many_passes():
    """More chunks than one pass's scratch holds: sequences cut at its border, one of them in place."""
    import ternary_weight_base_amd as tq
    heads, n = (64, 64, 128), [1300, 1500, 70, 1100]
    assert tq.tq_linear_attn_scratch_bytes(sum(n), 4, *heads) > 1 << 26
    c = make(heads, n, torch.float16, "heads", seed=10)
    c["to"][1] = c["from"][1]
    verify(c, *call(c))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=str)
def test_long_sequences(dtype):
    """More chunks than the scan's four runs of eight hold, and a sequence of one beside them."""
    for lengths in ([4500, 130], [1025, 1150], [2049, 1, 2170]):
        c = make((2, 1, 64), lengths, dtype, "rows", seed=18)
        verify(c, *call(c))


@pytest.mark.parametrize("seqs", [62, 63, 64, 65, 130])
def test_many_sequences_in_chunks(seqs):
    """Sequences found by a lane each, or searched for."""
    n = [(37 * i) % 61 + (200 if i % 29 == 5 else 0) for i in range(seqs)]
    n[-1] = 140
    c = make((2, 2, 64), n, torch.float16, "heads", seed=seqs)
    assert sum(n) > 16 * seqs
    verify(c, *call(c))


def test_sequences_across_two_borders_of_one_pass():
    """The second sequence ends in the pass that the third one is cut in: each has its own state between passes."""
    c = make((64, 64, 128), [2300, 2600, 600], torch.float16, "heads", seed=17)
    verify(c, *call(c))


def test_a_sequences_results_do_not_depend_on_the_others():
    """Nor on its cut into calls beyond the forms' rounding: chunks again from a state left behind."""
    c = make((8, 2, 64), [256, 300], torch.float16, "rows", seed=11)
    out, states = call(c)
    for s in range(2):
        one = dict(c)
        a, b = c["cu"][s], c["cu"][s + 1]
        one.update(qkv=c["qkv"][a:b], decay=c["decay"][a:b], cu=[0, b - a], **{"from": [c["from"][s]], "to": [c["to"][s]]})
        o, st = call(one)
        assert torch.equal(o, out[a:b]) and torch.equal(st[c["to"][s]], states[c["to"][s]])


def test_non_finite_rows_stay_with_their_sequence():
    for n in ([6, 5, 7], [200, 150, 260]):
        c = make((4, 2, 64), n, torch.float32, "rows", seed=12)
        clean, states = call(c)
        c["qkv"][c["cu"][1] + 2] = math.inf
        c["qkv"][c["cu"][1] + 4] = math.nan
        out, st = call(c)
        for s in (0, 2):
            a, b = c["cu"][s], c["cu"][s + 1]
            assert torch.equal(out[a:b], clean[a:b]) and torch.equal(st[c["to"][s]], states[c["to"][s]])


def test_bad_cu_rows_stay_inside():
    """Entries out of order or outside: wrong rows, no access outside the tensors."""
    for n in ([4, 2, 7], [200, 3, 150]):
        for cu in ([0, 5, 3, 13], [-7, 4, 1 << 30, 9], [0, 0, 0, 0], [5, 4, 3, 2]):
            c = make((4, 2, 64), n, torch.float16, "rows", seed=13)
            c["cu"] = cu
            call(c)


@pytest.mark.parametrize("n", [[1] * 6, [150, 40, 300]], ids=["rows", "chunks"])
def test_captured_with_changing_lengths(n):
    """One graph, replayed with other rows, lengths and states; eager calls between."""
    import ternary_weight_base_amd as tq
    heads = (8, 2, 64)
    c = make(heads, n, torch.float32, "rows", seed=14)
    rows, seqs = c["qkv"].shape[0], len(n)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu, start, to = dev(c["cu"]), dev(c["from"]), dev(c["to"])
    states, out = c["states"].clone(), torch.empty((rows, 8, 64), dtype=torch.float16, device="cuda")
    scratch = tq.linear_attn_scratch(rows, seqs, *heads)
    run = lambda: tq.tq_linear_attn(c["qkv"], c["decay"], cu, start, to, states, out, scratch=scratch)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        o = make(heads, n, torch.float32, "rows", seed=20 + i)
        lens = [max(0, x - i * (j + 1)) for j, x in enumerate(n)]
        o["cu"] = [sum(lens[:j]) for j in range(seqs + 1)]
        o["scale"] = 0.125
        c["qkv"].copy_(o["qkv"])
        c["decay"].copy_(o["decay"])
        states.copy_(o["states"])
        cu.copy_(dev(o["cu"]))
        start.copy_(dev(o["from"]))
        to.copy_(dev(o["to"]))
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want, st = call(o)
        a = o["cu"][-1]
        assert torch.equal(out[:a], want[:a]) and torch.equal(states, st)
        assert bool(torch.isnan(out[a:]).all())


def test_two_streams_with_scratch_of_their_own():
    cases = [make((8, 2, 64), [300, 200], torch.float16, "rows", seed=30 + i) for i in range(2)]
    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    import ternary_weight_base_amd as tq
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = [(c["qkv"], c["decay"], dev(c["cu"]), dev(c["from"]), dev(c["to"]), c["states"].clone(),
             torch.empty((500, 8, 64), dtype=torch.float16, device="cuda")) for c in cases]
    scratch = [tq.linear_attn_scratch(500, 2, 8, 2, 64) for _ in cases]
    torch.cuda.synchronize()
    for a, c, w, s in zip(args, cases, scratch, streams):
        tq.tq_linear_attn(*a, scale=c["scale"], scratch=w, stream=s)
        got.append(a)
    torch.cuda.synchronize()
    for a, (o, st) in zip(got, want):
        assert torch.equal(a[6], o) and torch.equal(a[5], st)
