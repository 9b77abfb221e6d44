"""A small model served with the calls as they are used together: a layer of
linear attention and one of attention over the cache, a prompt that all users
share, then steps of one token each, chosen from the logits.  Every new call's
results are held against its 64-bit reference on the inputs that it got, and the
whole step, captured once, against the eager steps."""
import numpy as np
import pytest

import linear_util
import sample_util
from gpu_util import B3, dev, upload_blob, weights
from kv_util import PAGE, attention, attention_tolerance

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

H, HQ, HKV, D, VOCAB = 512, 8, 2, 64, 16384
QKV, USERS, PROMPT, STEPS = (HQ + 2 * HKV) * D, 9, 2 * PAGE, 4
TOLD = 1 << 17  # the prefix as the attention is told of it: in a launch of its own
SHAPES = {"qkv1": (QKV, H), "o1": (H, HQ * D), "qkv2": (QKV, H), "o2": (H, HQ * D), "head": (VOCAB, H)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Model:
    def __init__(self, seed):
        import ternary_weight_base_amd as tq
        rng = np.random.default_rng(seed)
        self.w = {n: upload_blob(B3, *weights(*s, seed + i)) for i, (n, s) in enumerate(SHAPES.items())}
        self.emb = dev(rng.standard_normal((VOCAB, H)).astype(np.float32))
        self.norm = dev(1 + 0.1 * rng.standard_normal((3, H)).astype(np.float32))
        self.rope = dev(tq.tq_rope_table(PROMPT + 64, D, 10000.0))
        self.decay = dev(-np.linspace(0.01, 0.2, HKV, dtype=np.float32))
        nbytes = [tq.tq_gemm_workspace_bytes(B3, m, n, k) for n, k in SHAPES.values() for m in (PROMPT, USERS)]
        nbytes += [tq.tq_kv_attn_shared_workspace_bytes(USERS, USERS, 1, HQ, HKV, D, TOLD, 64), tq.tq_sample_workspace_bytes(USERS, VOCAB),
                   tq.tq_kv_attn_workspace_bytes(PROMPT, 1, HQ, HKV, D, PROMPT)]
        self.ws = torch.zeros(max(nbytes) // 4 + 4, dtype=torch.int32, device="cuda")  # one for all calls
        # users: temperature 0 (the largest), limits of each kind and all
        self.limits = dict(temperature=dev(np.array([0, 1, 1, 1, 1, 0.7, 1.5, 1, 0.9], np.float32)),
                           top_k=dev(np.array([0, 0, 40, 0, 0, 20, 1000, 1, 50], np.int32)),
                           top_p=dev(np.array([1, 1, 1, 0.9, 1, 0.95, 0.8, 1, 0.99], np.float32)),
                           min_p=dev(np.array([0, 0, 0, 0, 0.1, 0.02, 0, 0, 0.001], np.float32)))
        self.start()

    def start(self):
        """Before the prompt: pages of garbage, user u's own page behind the shared ones."""
        self.k, self.v = (torch.full(s, 77, dtype=torch.uint8, device="cuda") for s in
                          ((USERS + 3, HKV, PAGE, D), (USERS + 3, HKV, D, PAGE)))
        self.ks, self.vs = (torch.zeros((USERS + 3, HKV), device="cuda") for _ in range(2))
        self.states = torch.full((USERS + 1, HKV, D, D), 3.0, device="cuda")
        table = np.full((USERS, 4), -1, np.int32)
        table[:, :2] = [5, 1]
        table[:, 2] = [i for i in range(USERS + 3) if i not in (5, 1)][:USERS]
        self.table = dev(table)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.kv_len = torch.full((USERS,), PROMPT, **i32)
        self.token = torch.arange(USERS, **i32) * 7
        self.u, self.logprob = torch.zeros(USERS, device="cuda"), torch.zeros(USERS, device="cuda")
        self.cu = torch.arange(USERS + 1, **i32)
        self.cu_seqs, self.prefix = dev(np.array([0, USERS], np.int32)), dev(np.array([PROMPT], np.int32))
        self.own = torch.arange(1, USERS + 1, **i32)
        self.shared = torch.zeros(USERS, **i32)

    def gemm(self, name, q, a):
        import ternary_weight_base_amd as tq
        n, k = SHAPES[name]
        y = torch.empty((q.shape[0], n), device="cuda")
        tq.tq_gemm(B3, q.shape[0], n, k, self.w[name], q, a, y, ws=self.ws)
        return y

    def norm_to(self, i, y, res):
        import ternary_weight_base_amd as tq
        q, a = torch.empty(res.shape, dtype=torch.int8, device="cuda"), torch.empty(res.shape[0], device="cuda")
        out = None if y is None else torch.empty_like(res)
        tq.tq_residual_norm(y, res, out, pre_w=self.norm[i], q=q, a_scale=a)
        return (res if y is None else out), q, a

    def project(self, name, x):
        import ternary_weight_base_amd as tq
        q, a = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
        tq.tq_quant_act(x, q, a)
        return self.gemm(name, q, a)

    def layers(self, tokens, cu, table, kv_len, start, to, attend, see=None):
        """tokens' rows through both layers -> the last norm's codes; `see` gets each call's inputs and outputs."""
        import ternary_weight_base_amd as tq
        rows = tokens.shape[0]
        res, q, a = self.norm_to(0, None, self.emb.index_select(0, tokens))
        qkv = self.gemm("qkv1", q, a)
        out = torch.empty((rows, HQ, D), dtype=torch.float16, device="cuda")
        before = self.states.clone() if see is not None else None
        scratch = tq.linear_attn_scratch(rows, cu.shape[0] - 1, HQ, HKV, D)
        tq.tq_linear_attn(qkv, self.decay, cu, start, to, self.states, out, scratch=scratch)
        if see is not None:
            see.append(("linear", qkv, before, out, self.states.clone()))
        res, q, a = self.norm_to(1, self.project("o1", out.flatten(1)), res)
        qr, out = (torch.empty((rows, HQ, D), dtype=torch.float16, device="cuda") for _ in range(2))
        cache = (self.k, self.v, self.ks, self.vs)
        tq.tq_kv_append(self.gemm("qkv2", q, a), self.rope, cu, kv_len, table, *cache, q_out=qr)
        attend(qr, cache, out)
        if see is not None:
            see.append(("attention", qr, [t.clone() for t in cache], kv_len.clone(), out))
        return self.norm_to(2, self.project("o2", out.flatten(1)), res)

    def prompt(self, see=None):
        import ternary_weight_base_amd as tq
        cu, one = dev(np.array([0, PROMPT], np.int32)), self.table[:1].contiguous()
        none, first = dev(np.array([-1], np.int32)), dev(np.array([0], np.int32))
        def attend(q, cache, out):
            tq.tq_kv_attn(q, cu, self.kv_len[:1].contiguous(), one, *cache, out, PROMPT, ws=self.ws)
        _, q, a = self.layers(torch.arange(PROMPT, device="cuda") * 31 % VOCAB, cu, one, self.kv_len[:1].contiguous(), none, first, attend, see)
        self.gain = 3 / self.gemm("head", q, a).std()

    def step(self, first, see=None):
        """One token of all users; the first step starts from the prompt's state, later ones in place."""
        import ternary_weight_base_amd as tq
        self.kv_len.add_(1)
        def attend(q, cache, out):
            tq.tq_kv_attn_shared(q, self.cu, self.kv_len, self.cu_seqs, self.prefix, self.table, *cache, out, TOLD, 64, ws=self.ws)
        _, q, a = self.layers(self.token, self.cu, self.table, self.kv_len, self.shared if first else self.own, self.own, attend, see)
        logits = self.gemm("head", q, a)
        logits.mul_(self.gain)
        tq.tq_sample(logits, self.u, self.token, **self.limits, logprob=self.logprob, ws=self.ws)
        if see is not None:
            see.append(("sample", logits, self.u.clone(), self.token.clone(), self.logprob.clone()))

    def draw(self, step):
        self.u.copy_(dev(np.random.default_rng(step).random(USERS).astype(np.float32)))

    def held(self):
        return [t.clone() for t in (self.token, self.logprob, self.states, self.kv_len, self.k, self.v, self.ks, self.vs)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def run(m, see=None):
    """-> what each eager step leaves."""
    m.start()
    m.prompt(see)
    left = []
    for i in range(STEPS):
        m.draw(i)
        m.step(i == 0, see)
        left.append(m.held())
    return left


def test_each_call_against_its_reference():
    m, see = Model(70), []
    run(m, see)
    assert int(m.ws.count_nonzero()) == 0
    limits = {k: t.cpu().numpy() for k, t in m.limits.items()}
    table, steps = m.table.cpu().numpy(), {"linear": 0, "attention": 0, "sample": 0}
    for what, *x in see:
        i, steps[what] = steps[what], steps[what] + 1  # 0: the prompt (sample: the first step)
        cu = [0, PROMPT] if i == 0 else list(range(USERS + 1))
        if what == "linear":
            qkv, before, out, after = x
            own = list(range(1, USERS + 1))
            start, to = ([-1], [0]) if i == 0 else ([0] * USERS if i == 1 else own, own)
            linear_util.check(out, after, qkv, m.decay, cu, start, to, before, D ** -0.5, HQ, HKV, D)
        elif what == "attention":
            q, cache, kv_len, out = x
            q, kv_len, *cache = (t.cpu().numpy() for t in (q, kv_len, *cache))
            ref, mag, dot = attention(q, cu, kv_len, table[:len(kv_len)], *cache, D ** -0.5, 0, 0)
            err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
            assert (err <= attention_tolerance(ref, mag, dot, int(kv_len.max()) + 8, D)).all()
        else:
            logits, u, token, logprob = (t.cpu().numpy() for t in x)
            for r in range(USERS):
                t, lp, margin = sample_util.sample(logits[r], u[r], *(limits[n][r] for n in ("temperature", "top_k", "top_p", "min_p")))
                if margin > 1e-6:  # (ln of a quotient that is off by up to 2^-25, rounded to fp32)
                    assert token[r] == t and abs(logprob[r] - lp) <= 2.0 ** -24 * (abs(lp) + 1)
    assert steps == {"linear": STEPS + 1, "attention": STEPS + 1, "sample": STEPS}


def test_captured_steps_are_the_eager_ones():
    """The step as a graph, with eager calls on the same workspace between its replays."""
    m = Model(80)
    eager = run(m)
    assert same(eager[-1], run(m)[-1]), "two runs differ"
    m.start()
    m.prompt()
    m.draw(0)
    m.step(True)
    assert same(eager[0], m.held())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(False)
    for i in range(1, STEPS):
        m.draw(i)
        graph.replay()
        torch.cuda.synchronize()
        assert same(eager[i], m.held()), f"step {i}"
        m.project("o1", torch.ones((USERS, HQ * D), dtype=torch.float16, device="cuda"))
    assert int(m.ws.count_nonzero()) == 0


def test_two_models_on_two_streams():
    """Each with its own workspace, cache and states: results are those of one alone."""
    a, b = Model(90), Model(91)
    alone = [run(a)[-1], run(b)[-1]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for m in (a, b):
        m.start()
    torch.cuda.synchronize()
    for i in range(-1, STEPS):
        for m, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                if i < 0:
                    m.prompt()
                else:
                    m.draw(i)
                    m.step(i == 0)
    torch.cuda.synchronize()
    assert same(alone[0], a.held()) and same(alone[1], b.held())
