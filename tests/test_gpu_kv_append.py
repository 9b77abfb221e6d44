"""tq_kv_append: rotated queries and the cache's bytes and scales against a
plain 64-bit reference that quantises every token with its page's final scale
(so appending in pieces has to give what one append gives, bit for bit)."""
import numpy as np
import pytest

from gpu_util import dev, say
from kv_util import PAGE, Cache, append_rows, lay_out

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rope(positions, rot, base=10000.0):
    import ternary_weight_base_amd as tq
    return tq.tq_rope_table(positions, rot, base) if rot else None


class Pool:
    """A cache on the GPU, filled with garbage (NaN scales), beside its reference."""

    def __init__(self, pages, hkv, dim, rng):
        self.pages, self.hkv, self.dim = pages, hkv, dim
        self.k0 = rng.integers(0, 256, (pages, hkv, PAGE, dim), dtype=np.uint8)
        self.v0 = rng.integers(0, 256, (pages, hkv, dim, PAGE), dtype=np.uint8)
        self.k, self.v = dev(self.k0), dev(self.v0)
        self.ks = torch.full((pages, hkv), float("nan"), device="cuda")
        self.vs = torch.full((pages, hkv), float("nan"), device="cuda")
        self.ref = Cache(pages, hkv, dim)

    def check(self):
        torch.cuda.synchronize()
        for name, got, first, sc, store, token_last in (("k", self.k, self.k0, self.ks, self.ref.k, False),
                                                        ("v", self.v, self.v0, self.vs, self.ref.v, True)):
            want, ws = first.copy(), np.full((self.pages, self.hkv), np.nan, np.float32)
            got = got.cpu().numpy()
            for page in store:
                s, codes = self.ref.codes(store, page)
                ws[page] = s
                top = max(codes)
                for slot, c in codes.items():
                    if token_last:
                        want[page, :, :, slot] = c
                    else:
                        want[page, :, slot] = c
                if token_last:  # bytes behind the last token, and other pages, keep what they held
                    assert np.array_equal(got[page, :, :, top + 1:], first[page, :, :, top + 1:]), (name, page)
            assert np.array_equal(sc.cpu().numpy(), ws, equal_nan=True), f"{name} scales"
            assert np.array_equal(got, want), f"{name} codes: {np.argwhere(got != want)[:4]}"


def _append(pool, qkv, hq, rope, rot, pairs, cu, kv_len, table, q_out=True):
    import ternary_weight_base_amd as tq
    rows = qkv.shape[0]
    q = torch.full((rows, hq, pool.dim), 7.0, dtype=torch.float16, device="cuda") if q_out else None
    tq.tq_kv_append(qkv if torch.is_tensor(qkv) else dev(qkv), None if rope is None else dev(rope), dev(np.array(cu, np.int32)),
                    dev(np.array(kv_len, np.int32)), dev(table), pool.k, pool.v, pool.ks, pool.vs, q,
                    rope_mode=tq.TQ_ROPE_PAIRS if pairs else tq.TQ_ROPE_HALVES, q_heads=hq)
    host = qkv.cpu().numpy() if torch.is_tensor(qkv) else qkv
    ref = append_rows(pool.ref, host, hq, pool.hkv, pool.dim, rope, rot, pairs, cu, kv_len, table, pool.pages)
    if q_out:
        got = q.cpu().numpy()
        want = np.full_like(got, 7.0)  # padding rows stay as they were
        for r, x in ref.items():
            want[r] = x
        assert np.array_equal(got.view(np.uint16), want.view(np.uint16)), "rotated queries"


CASES = [
    # (hq, hkv, dim, rot, pairs, dtype, [(new rows, kv_len)...], padding rows)
    (8, 2, 128, 128, False, np.float32, [(1, 1)], 0),
    (8, 2, 128, 128, True, np.float16, [(1, 64), (1, 65), (1, 129)], 0),
    (3, 3, 64, 64, False, np.float32, [(64, 64), (0, 17), (130, 130)], 3),
    (4, 1, 64, 32, True, np.float32, [(7, 7), (0, 0), (200, 200), (1, 1)], 0),
    (10, 2, 128, 64, False, np.float16, [(65, 65), (63, 63), (5, 5)], 70),
    (5, 1, 128, 0, False, np.float32, [(33, 33)], 0),
    (2, 2, 64, 8, True, np.float16, [(9, 4)], 1),     # more rows than tokens: the first rows have no position
    (2, 1, 128, 128, False, np.float32, [(3, 0), (4, 4)], 0),
    (4, 2, 128, 64, True, np.float32, [(21, 70)] + [(0, 5)] * 7 + [(1, 65)], 0),   # few rows a sequence, but many in one
] + [
    (4, 2, 64, 64, False, np.float32, [(1 + i % 3, 1 + i % 3) for i in range(150)], 2),
    (4, 2, 128, 64, True, np.float32, [(21, 70)] + [(0, 5)] * 70 + [(1, 65)], 0),  # the kernel for few rows, with many in one sequence
    (4, 2, 128, 128, False, np.float16, [(4, 66 + i) for i in range(70)], 1),
    (4, 2, 64, 32, True, np.float16, [(130, 131)] + [(0, 9)] * 140, 3),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append_from_empty(i):
    hq, hkv, dim, rot, pairs, dtype, lens, pad = CASES[i]
    say(f"append case {i}: {CASES[i][:6]} {len(lens)} sequences")
    rng = np.random.default_rng(100 + i)
    kv_len = [t for _, t in lens]
    # sequences whose rows begin behind position 0 get their page's earlier tokens first
    before = [max(0, t - n) for n, t in lens]
    table, pages = lay_out(rng, kv_len)
    pool = Pool(pages, hkv, dim, rng)
    rope = _rope(max(kv_len + [1]), rot)
    width = (hq + 2 * hkv) * dim
    if any(before):
        cu = np.cumsum([0] + before)
        _append(pool, rng.standard_normal((cu[-1], width)).astype(dtype), hq, rope, rot, pairs, cu, before, table)
    cu = np.cumsum([0] + [n for n, _ in lens])
    x = (rng.standard_normal((cu[-1] + pad, width)) * np.exp(rng.standard_normal((cu[-1] + pad, 1)))).astype(dtype)
    _append(pool, x, hq, rope, rot, pairs, cu, kv_len, table)
    pool.check()


@pytest.mark.parametrize("dim,dtype", [(128, np.float32), (64, np.float16)])
def test_cache_does_not_depend_on_the_cuts(dim, dtype):
    """One sequence appended token by token, in odd pieces and at once."""
    say(f"append in pieces, dim {dim}")
    rng = np.random.default_rng(7)
    hq, hkv, total = 4, 2, 150
    rope = _rope(total, dim)
    # magnitudes that grow and fall by powers of two: scales grow within a page, some by more than 2^8
    mag = 2.0 ** rng.integers(-12, 3, (total, 1, 1))
    x = (rng.standard_normal((total, hq + 2 * hkv, dim)) * mag).astype(dtype)
    x[5:9] = 0
    x[64:70] = 0  # a page that starts with zeros
    x = x.reshape(total, -1)
    bytes_ = []
    for cuts in ([1] * total, [3, 61, 1, 64, 20, 1], [total]):
        table, pages = np.array([[2, 0, 1, -1]], np.int32), 3
        pool = Pool(pages, hkv, dim, np.random.default_rng(8))
        at = 0
        for n in cuts:
            _append(pool, x[at:at + n], hq, rope, dim, False, [0, n], [at + n], table, q_out=at % 2 == 0)
            at += n
        pool.check()
        bytes_.append((pool.k.cpu().numpy(), pool.v.cpu().numpy(), pool.ks.cpu().numpy(), pool.vs.cpu().numpy()))
    for b in bytes_[1:]:
        for p, q in zip(bytes_[0], b):
            assert np.array_equal(p.view(np.uint8), q.view(np.uint8))


@pytest.mark.parametrize("value", [0.0, 1.0, 127.99999, 128.0, -128.0, 1.4e-45, -1.4e-45, 1e-38, 3e38, -3.4e38])
def test_scales_at_the_edges(value):
    say(f"append of {value}")
    hq, hkv, dim = 1, 1, 64
    pool = Pool(1, hkv, dim, np.random.default_rng(1))
    x = np.zeros((2, 3 * dim), np.float32)
    x[0, dim + 5] = value
    x[1, 2 * dim:] = -value
    x[1, dim:2 * dim] = value * np.linspace(0, 1, dim, dtype=np.float32)
    _append(pool, x, hq, None, 0, False, [0, 2], [2], np.array([[0]], np.int32))
    pool.check()


def test_strided_rows_and_rewriting():
    """Rows of a wider buffer; a rejected token's slot written again."""
    say("append strided")
    rng = np.random.default_rng(3)
    hq, hkv, dim = 6, 2, 128
    wide = dev(rng.standard_normal((70, (hq + 2 * hkv) * dim + 24)).astype(np.float32))
    pool = Pool(3, hkv, dim, rng)
    table = np.array([[1, 2]], np.int32)
    rope = _rope(80, dim)
    _append(pool, wide[:, 16:-8][:, :(hq + 2 * hkv) * dim], hq, rope, dim, True, [0, 70], [70], table)
    pool.check()
    # positions 64..66 anew, from the page's start
    x = rng.standard_normal((3, (hq + 2 * hkv) * dim)).astype(np.float32)
    _append(pool, x, hq, rope, dim, True, [0, 3], [67], table)
    got = pool.k.cpu().numpy()
    scale, codes = pool.ref.codes(pool.ref.k, 2)
    assert np.array_equal(pool.ks.cpu().numpy()[2], scale.astype(np.float32))
    for slot in range(3):
        assert np.array_equal(got[2, :, slot], codes[slot])


def test_bad_pages_and_positions_are_left_out():
    """Pages outside the pool, behind the table, and positions behind the rope
    table: not stored, nothing else touched; their queries: only the positions'."""
    say("append with bad pages")
    rng = np.random.default_rng(5)
    hq, hkv, dim = 2, 1, 64
    kv_len = [130, 70, 200, 66]
    table = np.array([[0, -1, 1], [2, 1 << 30, -7], [3, 4, 5], [-5, 6, 99]], np.int32)
    pool = Pool(8, hkv, dim, rng)
    rope = _rope(150, dim)
    cu = np.cumsum([0] + kv_len)
    x = rng.standard_normal((cu[-1], 4 * dim)).astype(np.float32)
    _append(pool, x, hq, rope, dim, False, cu, kv_len, table)
    pool.check()


def test_read_back():
    import ternary_weight_base_amd as tq
    say("read back")
    rng = np.random.default_rng(6)
    for dim, hkv in ((128, 2), (64, 3)):
        k = rng.integers(0, 256, (5, hkv, PAGE, dim), dtype=np.uint8)
        v = rng.integers(0, 256, (5, hkv, dim, PAGE), dtype=np.uint8)
        ks, vs = (2.0 ** rng.integers(-9, 3, (5, hkv))).astype(np.float32), rng.uniform(0.1, 3, (5, hkv)).astype(np.float32)
        ids = np.array([3, 0, 9, -1, 3], np.int32)
        for t in (torch.float32, torch.float16):
            out = torch.empty((2, 5, hkv, PAGE, dim), dtype=t, device="cuda")
            tq.tq_debug_kv_read(dev(ids), dev(k), dev(v), dev(ks), dev(vs), out)
            want = np.zeros((2, 5, hkv, PAGE, dim), np.float32)
            for i, p in enumerate(ids):
                if 0 <= p < 5:
                    want[0, i] = (k[p].astype(np.float32) - np.float32(127.5)) * ks[p][:, None, None]
                    want[1, i] = ((v[p].astype(np.float32) - np.float32(127.5)) * vs[p][:, None, None]).transpose(0, 2, 1)
            assert np.array_equal(out.cpu().numpy(), want.astype(out.cpu().numpy().dtype))


def test_graph_replay_with_new_lengths():
    """Captured once; lengths, rows and table change between the replays."""
    import ternary_weight_base_amd as tq
    say("append in a graph")
    rng = np.random.default_rng(9)
    hq, hkv, dim, seqs = 4, 2, 128, 3
    pool = Pool(12, hkv, dim, rng)
    table = rng.permutation(12).reshape(3, 4).astype(np.int32)
    rope = _rope(300, dim)
    d = {"x": torch.zeros((seqs, (hq + 2 * hkv) * dim), device="cuda"), "cu": dev(np.arange(seqs + 1, dtype=np.int32)),
         "kv": dev(np.zeros(seqs, np.int32)), "table": dev(table), "rope": dev(rope),
         "q": torch.zeros((seqs, hq, dim), dtype=torch.float16, device="cuda")}

    def call():
        tq.tq_kv_append(d["x"], d["rope"], d["cu"], d["kv"], d["table"], pool.k, pool.v, pool.ks, pool.vs, d["q"])

    call()  # no sequence has a token: nothing is stored
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.synchronize()
    junk = torch.randn(1 << 18, device="cuda")
    for step in range(1, 68):
        x = rng.standard_normal((seqs, (hq + 2 * hkv) * dim)).astype(np.float32)
        kv = [step, step, step]
        d["x"].copy_(torch.from_numpy(x))
        d["kv"].copy_(torch.tensor(kv, dtype=torch.int32))
        junk.mul_(1.0001)
        g.replay()
        torch.cuda.synchronize()
        ref = append_rows(pool.ref, x, hq, hkv, dim, rope, dim, False, np.arange(seqs + 1), kv, table, 12)
        got = d["q"].cpu().numpy()
        for r, q in ref.items():
            assert np.array_equal(got[r].view(np.uint16), q.view(np.uint16)), (step, r)
    pool.check()
