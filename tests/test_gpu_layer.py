"""A decoder layer run with the library's calls alone: norm -> QKV -> append ->
attention -> O -> norm -> gate/up/SwiGLU -> down -> norm, first a prompt of
two sequences, then single tokens, eager and from one captured graph.  Every
stage is checked against its 64-bit reference on the stage's own input."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import B3, assert_close, dev, say, upload_blob, weights
from kv_util import PAGE, Cache, append_rows, attention, attention_tolerance, norm

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

H, INTER, HQ, HKV, D = 640, 1152, 4, 2, 64
QKV = (HQ + 2 * HKV) * D
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    oracle.set_threads(8)


class Layer:
    def __init__(self, seed, pages, seqs, width):
        import ternary_weight_base_amd as tq
        self.shapes = {"qkv": (QKV, H), "o": (H, HQ * D), "gate": (INTER, H), "up": (INTER, H), "down": (H, INTER)}
        self.host = {n: weights(N, K, seed + i) for i, (n, (N, K)) in enumerate(self.shapes.items())}
        self.w = {n: upload_blob(B3, *tw) for n, tw in self.host.items()}
        rng = np.random.default_rng(seed)
        self.norms_host = [rng.uniform(0.5, 1.5, H).astype(np.float32) for _ in range(5)]
        self.norms = [dev(x) for x in self.norms_host]
        self.gate_host = rng.uniform(-1, 1, H).astype(np.float32)
        self.gate = dev(self.gate_host)
        self.rope_host = tq.tq_rope_table(width * PAGE, D, 1e4)
        self.rope = dev(self.rope_host)
        self.k = torch.zeros((pages, HKV, PAGE, D), dtype=torch.uint8, device="cuda")
        self.v = torch.zeros((pages, HKV, D, PAGE), dtype=torch.uint8, device="cuda")
        self.ks, self.vs = torch.zeros((pages, HKV), device="cuda"), torch.zeros((pages, HKV), device="cuda")
        self.table_host = rng.permutation(pages)[:seqs * width].reshape(seqs, width).astype(np.int32)
        self.table = dev(self.table_host)
        need = [tq.tq_kv_attn_workspace_bytes(seqs, seqs, HQ, HKV, D, width * PAGE)]
        need += [tq.tq_gemv_workspace_bytes(B3, seqs, N, K) for N, K in self.shapes.values()]
        self.ws = torch.zeros(max(need) // 4 + 4, dtype=torch.int32, device="cuda")

    def buffers(self, rows):
        f = dict(dtype=torch.float32, device="cuda")
        return {"res": torch.empty((rows, H), **f), "q1": torch.empty((rows, H), dtype=torch.int8, device="cuda"), "a1": torch.empty(rows, **f),
                "qkv": torch.empty((rows, QKV), **f), "q": torch.empty((rows, HQ, D), dtype=torch.float16, device="cuda"),
                "att": torch.empty((rows, HQ, D), dtype=torch.float16, device="cuda"),
                "q2": torch.empty((rows, HQ * D), dtype=torch.int8, device="cuda"), "a2": torch.empty(rows, **f),
                "y_o": torch.empty((rows, H), **f), "res2": torch.empty((rows, H), **f),
                "q3": torch.empty((rows, H), dtype=torch.int8, device="cuda"), "a3": torch.empty(rows, **f),
                "h": torch.empty((rows, INTER), **f), "q4": torch.empty((rows, INTER), dtype=torch.int8, device="cuda"),
                "a4": torch.empty(rows, **f), "y": torch.empty((rows, H), **f), "res3": torch.empty((rows, H), **f),
                "x": torch.empty((rows, H), dtype=torch.float16, device="cuda")}

    def attend(self, b, cu, kv, most):
        import ternary_weight_base_amd as tq
        rows = b["res"].shape[0]
        mm = (lambda n, q, a, y: tq.tq_gemv(B3, rows, *self.shapes[n], self.w[n], q, a, y, self.ws)) if rows <= 16 else \
            (lambda n, q, a, y: tq.tq_gemm(B3, rows, *self.shapes[n], self.w[n], q, a, y, tq.workspace(B3, rows, *self.shapes[n])))
        tq.tq_residual_norm(None, b["res"], None, self.norms[0], q=b["q1"], a_scale=b["a1"], eps=EPS)
        mm("qkv", b["q1"], b["a1"], b["qkv"])
        tq.tq_kv_append(b["qkv"], self.rope, cu, kv, self.table, self.k, self.v, self.ks, self.vs, b["q"])
        ws = self.ws if rows <= 16 else tq.kv_attn_workspace(rows, kv.numel(), HQ, HKV, D, most)
        tq.tq_kv_attn(b["q"], cu, kv, self.table, self.k, self.v, self.ks, self.vs, b["att"], most, ws=ws)
        tq.tq_quant_act(b["att"].view(rows, HQ * D), b["q2"], b["a2"])
        mm("o", b["q2"], b["a2"], b["y_o"])

    def token(self, b, cu, kv, most):
        import ternary_weight_base_amd as tq
        rows = b["res"].shape[0]
        self.attend(b, cu, kv, most)
        tq.tq_residual_norm(b["y_o"], b["res"], b["res2"], self.norms[2], q=b["q3"], a_scale=b["a3"], post_w=self.norms[1], gate=self.gate,
                            res_scale=0.5, eps=EPS)
        tq.tq_gemv_gate_up_swiglu(B3, rows, INTER, H, self.w["gate"], self.w["up"], b["q3"], b["a3"], b["h"], self.ws)
        tq.tq_quant_act(b["h"], b["q4"], b["a4"])
        tq.tq_gemv(B3, rows, H, INTER, self.w["down"], b["q4"], b["a4"], b["y"], self.ws)
        tq.tq_residual_norm(b["y"], b["res2"], b["res3"], self.norms[4], x=b["x"], post_w=self.norms[3], res_scale=0.5, eps=EPS)

    def check(self, b, cache, cu, kv, full):
        torch.cuda.synchronize()
        g = {n: t.cpu().numpy() for n, t in b.items()}
        _, x = norm(None, g["res"], None, None, None, 0, self.norms_host[0], EPS)
        deq = g["q1"] * g["a1"][:, None]
        assert np.abs(deq - x).max() <= 0.5001 * g["a1"].max()  # half a code
        t, s = self.host["qkv"]
        assert_close(g["qkv"], oracle.gemv(t, s, g["q1"], g["a1"]), "qkv")
        rot = append_rows(cache, g["qkv"], HQ, HKV, D, self.rope_host, D, False, cu, kv, self.table_host, self.k.shape[0])
        for r, q in rot.items():
            assert np.array_equal(g["q"][r].view(np.uint16), q.view(np.uint16))
        k, v, ks, vs = (z.cpu().numpy() for z in (self.k, self.v, self.ks, self.vs))
        for store, codes, sc, last in ((cache.k, k, ks, False), (cache.v, v, vs, True)):
            for page in store:
                want_s, want = cache.codes(store, page)
                assert np.array_equal(sc[page], want_s.astype(np.float32))
                for slot, c in want.items():
                    assert np.array_equal(codes[page, :, :, slot] if last else codes[page, :, slot], c)
        ref, mag, dot = attention(g["q"], cu, np.array(kv), self.table_host, k, v, ks, vs, D ** -0.5, 0, 0)
        assert np.all(np.abs(g["att"].astype(np.float64) - ref) <= attention_tolerance(ref, mag, dot, max(kv), D))
        t, s = self.host["o"]
        assert_close(g["y_o"], oracle.gemv(t, s, g["q2"], g["a2"]), "o")
        if not full:
            return
        r, x = norm(g["y_o"], g["res"], np.float32, self.norms_host[1], self.gate_host, 0.5, self.norms_host[2], EPS)
        assert_close(g["res2"], r, "residual")
        assert np.abs(g["q3"] * g["a3"][:, None] - x).max() <= 0.5001 * g["a3"].max()
        ref_h = oracle.swiglu(*(oracle.gemv(*self.host[n], g["q3"], g["a3"]) for n in ("gate", "up")))
        assert np.abs(g["h"] - ref_h).max() <= 1e-3 * np.abs(ref_h).max()
        assert_close(g["y"], oracle.gemv(*self.host["down"], g["q4"], g["a4"]), "down")
        r, x = norm(g["y"], g["res2"], np.float32, self.norms_host[3], None, 0.5, self.norms_host[4], EPS)
        assert_close(g["res3"], r, "residual behind the FFN")
        assert np.all(np.abs(g["x"] - x) <= 2.0 ** -10 * np.abs(x) + 2.0 ** -24)


def _prompt(L, cache, rng):
    lens = [70, 33]
    cu = np.array([0, 70, 103], np.int32)
    b = L.buffers(103)
    b["res"].copy_(torch.from_numpy(rng.standard_normal((103, H)).astype(np.float32)))
    L.attend(b, dev(cu), dev(np.array(lens, np.int32)), 70)
    L.check(b, cache, cu, lens, False)
    return lens


def test_layer_prompt_then_tokens():
    say("decoder layer")
    rng = np.random.default_rng(11)
    L = Layer(500, 8, 2, 3)
    cache = Cache(8, HKV, D)
    lens = _prompt(L, cache, rng)
    b, cu = L.buffers(2), np.array([0, 1, 2], np.int32)
    for step in range(3):
        lens = [x + 1 for x in lens]
        b["res"].copy_(torch.from_numpy(rng.standard_normal((2, H)).astype(np.float32)))
        L.token(b, dev(cu), dev(np.array(lens, np.int32)), max(lens))
        L.check(b, cache, cu, lens, True)
    assert int(torch.count_nonzero(L.ws)) == 0


def test_layer_token_from_a_graph():
    """One captured step replayed for several tokens, the lengths counted up
    on the device: the same bits as the eager calls."""
    say("decoder layer in a graph")
    results = []
    for graph in (False, True):
        rng = np.random.default_rng(12)
        L = Layer(600, 8, 2, 3)
        lens = _prompt(L, Cache(8, HKV, D), rng)
        b, cu, kv = L.buffers(2), dev(np.array([0, 1, 2], np.int32)), dev(np.array(lens, np.int32))
        most = 3 * PAGE  # room for every length of the run
        call = lambda: (kv.add_(1), L.token(b, cu, kv, most))
        if graph:
            saved = [t.clone() for t in (L.k, L.v, L.ks, L.vs, kv)]
            b["res"].zero_()
            call()  # (the first call outside the capture)
            torch.cuda.synchronize()
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    call()
            torch.cuda.synchronize()
            for t, old in zip((L.k, L.v, L.ks, L.vs, kv), saved):
                t.copy_(old)
        outs = []
        for step in range(60):
            b["res"].copy_(torch.from_numpy(rng.standard_normal((2, H)).astype(np.float32)))
            torch.cuda.synchronize()
            g.replay() if graph else call()
            torch.cuda.synchronize()
            outs.append((b["x"].cpu().numpy().copy(), b["att"].cpu().numpy().copy()))
        assert kv.cpu().tolist() == [x + 60 for x in lens]
        results.append((outs, [t.cpu().numpy() for t in (L.k, L.v, L.ks, L.vs)]))
    for (x0, a0), (x1, a1) in zip(results[0][0], results[1][0]):
        assert np.array_equal(x0.view(np.uint16), x1.view(np.uint16)) and np.array_equal(a0.view(np.uint16), a1.view(np.uint16))
    for p, q in zip(results[0][1], results[1][1]):
        assert np.array_equal(p, q)


def test_layer_tokens_with_cut_keys_share_the_workspace():
    """Tokens on contexts long enough that attention's keys are cut: it and the
    projections take one workspace in turn, eager and replayed."""
    import ternary_weight_base_amd as tq
    say("decoder layer, attention in pieces")
    rng = np.random.default_rng(13)
    width = 20
    L = Layer(700, 2 * width, 2, width)
    assert tq.tq_kv_attn_workspace_bytes(2, 2, HQ, HKV, D, width * PAGE) > 0
    cache = Cache(2 * width, HKV, D)
    lens = _prompt(L, cache, rng)
    b, cu, kv = L.buffers(2), np.array([0, 1, 2], np.int32), dev(np.array(lens, np.int32))
    call = lambda: (kv.add_(1), L.token(b, dev_cu, kv, width * PAGE))
    dev_cu = dev(cu)
    graph = None
    for step in range(6):
        lens = [x + 1 for x in lens]
        b["res"].copy_(torch.from_numpy(rng.standard_normal((2, H)).astype(np.float32)))
        if step == 3:
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    call()
        torch.cuda.synchronize()
        graph.replay() if graph else call()
        L.check(b, cache, cu, lens, True)
        assert int(torch.count_nonzero(L.ws)) == 0
