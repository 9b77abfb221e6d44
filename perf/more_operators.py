"""What a server's step needs beside the cache, attention and norm calls, and the cases it is measured on.

  linear  tq_linear_attn: linear attention with a decay for each head and a recurrent state (prompts and single tokens)
  shared  tq_kv_attn_shared: attention over the paged 8-bit cache for groups of sequences that share a long prefix
  sample  tq_sample: the next token by temperature, top-k, top-p and min-p from given random numbers

The cache holds a byte b as the value (b - 127.5) * s with one power-of-two scale s for each page of 64 tokens and
KV head: K as [pages][heads][64][dim], V as [pages][heads][dim][64].
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
CHUNK = 64  # rows that the plain linear attention takes at once
# (query heads, KV heads, head dim); the first is this repository's 27B-shaped layer (QKV 5120 -> 10240)
HEADS = ((64, 8, 128), (32, 8, 128), (40, 8, 128), (16, 16, 64), (24, 4, 64))


def _heads(h):
    return {"q_heads": h[0], "kv_heads": h[1], "dim": h[2]}


def listed():
    a, b, c, d = HEADS[0], HEADS[1], HEADS[2], HEADS[3]
    return [
        # one user's next token: the whole call is latency
        {"name": "linear_1", "op": "linear", **_heads(a), "seqs": 1, "rows": 1, "ragged": False, "dtype": "f32", "decay": "rows",
         "fresh": False},
        # a server's step: 64 users, one token each, fp16 projections: the states' traffic
        {"name": "linear_64", "op": "linear", **_heads(b), "seqs": 64, "rows": 1, "ragged": False, "dtype": "f16", "decay": "rows",
         "fresh": False},
        # four drafted tokens for each of 8 users, their states written beside the old ones, a KV head a query head
        {"name": "linear_drafts", "op": "linear", **_heads(d), "seqs": 8, "rows": 4, "ragged": True, "dtype": "f32", "decay": "heads",
         "fresh": False},
        # a prompt of 4096 tokens from the projections' fp32
        {"name": "linear_prompt", "op": "linear", **_heads(a), "seqs": 1, "rows": 4096, "ragged": False, "dtype": "f32",
         "decay": "rows", "fresh": True},
        # pieces of three prompts of different lengths that go on from earlier states
        {"name": "linear_packed", "op": "linear", **_heads(d), "seqs": 3, "rows": 2051, "ragged": True, "dtype": "f16",
         "decay": "heads", "fresh": False},
        # eight users behind one system prompt, a short chat each
        {"name": "shared_8", "op": "shared", **_heads(a), "groups": 1, "seqs": 8, "rows": 1, "prefix": 2048, "own": 301, "ragged": True},
        # a server's step: 64 users behind a long one
        {"name": "shared_64", "op": "shared", **_heads(a), "groups": 1, "seqs": 64, "rows": 1, "prefix": 16384, "own": 1001,
         "ragged": True},
        # four system prompts of different lengths, users unevenly over them, two drafted tokens each
        {"name": "shared_groups", "op": "shared", **_heads(c), "groups": 4, "seqs": 37, "rows": 2, "prefix": 8000, "own": 777,
         "ragged": True},
        # sixteen users' first questions arrive at once behind one system prompt
        {"name": "shared_prompts", "op": "shared", **_heads(b), "groups": 1, "seqs": 16, "rows": 150, "prefix": 4096, "own": 203,
         "ragged": True},
        # one user's next token: latency
        {"name": "sample_1", "op": "sample", "rows": 1, "vocab": 131072, "dtype": "f32", "filters": "all"},
        # a server's step, every user with settings of its own
        {"name": "sample_64", "op": "sample", "rows": 64, "vocab": 131072, "dtype": "f32", "filters": "mixed"},
        # fp16 logits of an odd vocabulary (many ties), temperature alone
        {"name": "sample_odd", "op": "sample", "rows": 7, "vocab": 50001, "dtype": "f16", "filters": "none"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "shared", "shared", "sample"))
    if op == "sample":
        return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 1000, 131072), "dtype": rng.choice(("f16", "f32")),
                "filters": rng.choice(("all", "mixed", "none", "k", "p"))}
    c = {"op": op, **_heads(rng.choice(HEADS))}
    many = rng.random() < 0.4
    if op == "linear":
        c |= {"seqs": rng.randint(1, 3), "rows": _log(rng, 17, 2000)} if many else \
            {"seqs": _log(rng, 1, 64), "rows": rng.choice((1, 1, 2, 3, 4, 9))}
        c |= {"dtype": rng.choice(("f16", "f32")), "decay": rng.choice(("heads", "rows")), "fresh": rng.random() < 0.4}
    else:
        c |= {"seqs": _log(rng, 2, 16), "rows": _log(rng, 5, 200)} if many else {"seqs": _log(rng, 2, 64), "rows": rng.choice((1, 1, 2, 4))}
        c |= {"groups": min(c["seqs"], rng.choice((1, 1, 2, 4))), "prefix": _log(rng, 128, 8192), "own": c["rows"] + _log(rng, 1, 1000)}
    c["ragged"] = rng.random() < 0.7
    while c["seqs"] > 2 and (work(c)["flops"] > 3.5e10 or work(c)["bytes"] > 2.4e8):
        c["seqs"] -= 1
        if op == "shared":
            c["groups"] = min(c["groups"], c["seqs"])
    return c


DTYPES = {"f16": torch.float16, "f32": torch.float32}


def _rows(case):
    """New rows of each sequence: spread below the case's largest where it is ragged."""
    r = random.Random("%(seqs)d %(rows)d" % case)
    return [case["rows"] if s == 0 or not case["ragged"] else r.randint((case["rows"] + 1) // 2, case["rows"]) for s in range(case["seqs"])]


def _sharing(case):
    """(new rows, own tokens) of each sequence, (sequences, prefix) of each group."""
    n = _rows(case)
    r = random.Random("%(seqs)d %(own)d %(prefix)d" % case)
    own_tokens = [case["own"] if s == 0 or not case["ragged"] else max(n[s], r.randint(case["own"] // 4, case["own"]))
                  for s in range(case["seqs"])]
    g = case["groups"]
    cuts = sorted(r.sample(range(1, case["seqs"]), g - 1))
    members = [b - a for a, b in zip([0] + cuts, cuts + [case["seqs"]])]
    most = case["prefix"] // PAGE
    prefix = [PAGE * (most if i == 0 or not case["ragged"] else r.randint(most // 4, most)) for i in range(g)]
    return n, own_tokens, members, prefix


def _starts(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _device(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _prepare_linear(case, g):
    n = _rows(case)
    rows, seqs, hq, hkv, dim = sum(n), case["seqs"], case["q_heads"], case["kv_heads"], case["dim"]
    st = {"case": case, "cu": _device(_starts(n)), "total": rows}
    st["qkv"] = torch.randn((rows, (hq + 2 * hkv) * dim), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    if case["decay"] == "heads":  # from a few tokens of memory to thousands, as fixed decays are laid out
        i = torch.arange(1, hkv + 1, device="cuda") / hkv
        st["decay"] = -torch.exp2(-1 - 10 * i) * (0.9 + 0.2 * torch.rand(hkv, generator=g, device="cuda"))
    else:  # gates of the rows: mostly near one, now and then nearly shut
        x = 2 * torch.randn((rows, hkv), generator=g, device="cuda") + 4
        st["decay"] = -torch.log1p(torch.exp(-x))
    # states are read from the first half of the pool and written to the second, as a server forks or keeps them
    st["states"] = torch.randn((2 * seqs, hkv, dim, dim), generator=g, device="cuda") * 3
    order = torch.randperm(seqs, generator=g, device="cuda").int()
    st["from"] = torch.full_like(order, -1) if case["fresh"] else order
    st["to"] = seqs + order
    st["out"] = torch.zeros((rows, hq, dim), dtype=torch.float16, device="cuda")
    return st


def _prepare_shared(case, g):
    n, own_tokens, members, prefix = _sharing(case)
    heads, dim, rows = case["kv_heads"], case["dim"], sum(n)
    shared = [p // PAGE for p in prefix]
    used = [-(-t // PAGE) for t in own_tokens]
    pages = sum(shared) + sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    group = [i for i, m in enumerate(members) for _ in range(m)]
    width = max(shared[group[s]] + used[s] for s in range(case["seqs"]))
    table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")  # no page where a sequence has ended
    at, first = sum(shared), _starts(shared)
    for s, u in enumerate(used):
        p = shared[group[s]]
        table[s, :p] = order[first[group[s]]:first[group[s]] + p]
        table[s, p:p + u] = order[at:at + u]
        at += u

    def codes(*shape):
        # normal values, their largest using the upper half of the bytes' range, as a power-of-two scale leaves it
        spread = 28 * (0.5 + 0.5 * torch.rand((pages, heads, 1, 1), generator=g, device="cuda"))
        x = torch.randn(shape, generator=g, device="cuda").mul_(spread).add_(128).floor_().clamp_(0, 255)
        return x.to(torch.uint8)

    def scales():
        e = torch.randint(-6, -3, (pages, heads), generator=g, device="cuda").int()
        return ((e + 127) << 23).view(torch.float32)  # powers of two

    q = (2 * torch.randn((rows, case["q_heads"], dim), generator=g, device="cuda")).half()
    return {"case": case, "cu": _device(_starts(n)), "kv": _device([prefix[group[s]] + t for s, t in enumerate(own_tokens)]),
            "cu_seqs": _device(_starts(members)), "prefix": _device(prefix), "table": table, "total": rows, "most_prefix": max(prefix),
            "most_own": max(own_tokens), "k": codes(pages, heads, PAGE, dim), "v": codes(pages, heads, dim, PAGE), "ks": scales(),
            "vs": scales(), "q": q, "out": torch.zeros_like(q)}


def _prepare_sample(case, g):
    rows, vocab = case["rows"], case["vocab"]
    x = 2.2 * torch.randn((rows, vocab), generator=g, device="cuda")
    likely = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")  # what the context asks for
    x.scatter_add_(1, likely, 4 + 6 * torch.rand((rows, 40), generator=g, device="cuda"))
    x[:, vocab - vocab // 50:] = -math.inf  # tokens that may not come
    st = {"case": case, "logits": x.to(DTYPES[case["dtype"]]), "u": torch.rand(rows, generator=g, device="cuda")}
    r = random.Random("%(rows)d %(vocab)d %(filters)s" % case)
    f = case["filters"]
    st["temperature"] = _device([r.choice((0.6, 0.8, 1.0, 1.3)) if f != "mixed" or r.random() < 0.9 else 0.0 for _ in range(rows)],
                                torch.float32)
    st["top_k"] = st["top_p"] = st["min_p"] = None
    if f in ("all", "mixed", "k"):
        st["top_k"] = _device([r.choice((20, 50, 400)) if f != "mixed" else r.choice((0, 0, 1, 40, 1000)) for _ in range(rows)])
    if f in ("all", "mixed", "p"):
        st["top_p"] = _device([r.choice((0.8, 0.9, 0.95)) if f != "mixed" else r.choice((1.0, 0.95, 0.5)) for _ in range(rows)],
                              torch.float32)
    if f in ("all", "mixed"):
        st["min_p"] = _device([0.02 if f != "mixed" else r.choice((0.0, 0.0, 0.05)) for _ in range(rows)], torch.float32)
    st["token"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    st["logprob"] = torch.zeros(rows, device="cuda")
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"linear": _prepare_linear, "shared": _prepare_shared, "sample": _prepare_sample}[case["op"]](case, g)


def _linear_plain(st):
    case = st["case"]
    seqs, hq, hkv, dim = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"]
    n, group, scale = case["rows"], hq // hkv, dim ** -0.5
    cu = st["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=st["total"] - 1)
    there = i < count[:, None]
    x = st["qkv"][row].float().view(seqs, n, hq + 2 * hkv, dim) * there[..., None, None]
    q = x[:, :, :hq].reshape(seqs, n, hkv, group, dim).permute(0, 2, 3, 1, 4)
    k = x[:, :, hq:hq + hkv].transpose(1, 2)
    v = x[:, :, hq + hkv:].transpose(1, 2)
    d = st["decay"].double().expand(st["total"], hkv)[row] * there[..., None]
    start = st["from"].long()
    state = st["states"][start.clamp(min=0)] * (start >= 0)[:, None, None, None]
    out = torch.empty((seqs, hkv, group, n, dim), device="cuda")
    for c in range(0, n, CHUNK):
        m = min(CHUNK, n - c)
        run_ = d[:, c:c + m].cumsum(1).transpose(1, 2)  # [seqs][hkv][m]
        qc = q[:, :, :, c:c + m].reshape(seqs, hkv, group * m, dim)
        kc, vc = k[:, :, c:c + m], v[:, :, c:c + m]
        late = torch.ones((m, m), device="cuda").tril()
        w = (run_[..., :, None] - run_[..., None, :]).clamp(max=0).exp().float() * late
        p = torch.matmul(qc, kc.transpose(2, 3).contiguous()).view(seqs, hkv, group, m, m) * w[:, :, None]
        o = torch.matmul(p.view(seqs, hkv, group * m, m), vc.contiguous())
        o = o.view(seqs, hkv, group, m, dim) + torch.matmul(qc, state).view(seqs, hkv, group, m, dim) * run_.exp().float()[:, :, None, :, None]
        out[:, :, :, c:c + m] = scale * o
        left = (run_[..., -1:] - run_).exp().float()
        state = state * run_[..., -1].exp().float()[..., None, None] + torch.matmul((kc * left[..., None]).transpose(2, 3).contiguous(),
                                                                                     vc.contiguous())
    st["states"][st["to"].long()] = state
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(seqs, n, hq, dim).half()[there], "states": st["states"]}


def _values(st, ids):
    """Keys and values [heads][tokens][dim] in fp32 of the pages ids."""
    heads, dim = st["k"].shape[1], st["k"].shape[3]
    k = (st["k"][ids].float() - 127.5) * st["ks"][ids][..., None, None]
    v = (st["v"][ids].float() - 127.5) * st["vs"][ids][..., None, None]
    return k.transpose(0, 1).reshape(heads, -1, dim), v.permute(1, 0, 3, 2).reshape(heads, -1, dim)


def _shared_plain(st):
    case = st["case"]
    n, own_tokens, members, prefix = _sharing(case)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    group, cu, scale = hq // hkv, _starts(n), dim ** -0.5
    out = torch.empty((st["total"], hq, dim), device="cuda")
    s = 0
    for m, p in zip(members, prefix):
        # the prefix, once for all rows of the group
        a, b = cu[s], cu[s + m]
        q = st["q"][a:b].float().view(b - a, hkv, group, dim).transpose(0, 1)  # [hkv][rows][group][dim]
        kp, vp = _values(st, st["table"][s, :p // PAGE].long())
        before = torch.matmul(q.reshape(hkv, -1, dim), kp.transpose(1, 2).contiguous()).view(hkv, b - a, group, p) * scale
        for i in range(s, s + m):
            r = slice(cu[i] - a, cu[i + 1] - a)
            t = own_tokens[i]
            ko, vo = _values(st, st["table"][i, p // PAGE:p // PAGE - (-t // PAGE)].long())
            score = torch.matmul(q[:, r].reshape(hkv, -1, dim), ko[:, :t].transpose(1, 2).contiguous()).view(hkv, n[i], group, t) * scale
            hide = torch.arange(t, device="cuda") > torch.arange(t - n[i], t, device="cuda")[:, None]
            z = torch.cat((before[:, r], score.masked_fill_(hide[:, None], -math.inf)), -1)
            w = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(w.view(hkv, -1, p + t), torch.cat((vp, vo[:, :t]), 1)).view(hkv, n[i], group, dim)
            out[cu[i]:cu[i + 1]] = (o / w.sum(-1, keepdim=True)).transpose(0, 1).reshape(n[i], hq, dim)
        s += m
    return out.half()


def _sample_plain(st):
    # in 64 bits: a token's place in the running sum decides
    rows, vocab = st["logits"].shape
    x = st["logits"].double()
    t = st["temperature"].double()[:, None]
    best = x.amax(1, keepdim=True)
    z = (x - best) / torch.where(t > 0, t, 1)
    z, order = torch.sort(z, dim=1, descending=True, stable=True)  # ties: the lowest index first
    w = z.exp()
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        w = w * (torch.arange(vocab, device="cuda") < torch.where(k > 0, k, vocab))
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        run_ = w.cumsum(1)
        w = torch.where((p >= 1) | (run_ - w < p * run_[:, -1:]) | (torch.arange(vocab, device="cuda") == 0), w, 0)
    if st["min_p"] is not None:
        w = torch.where(w >= st["min_p"].double()[:, None], w, 0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    run_ = w.cumsum(1)
    total = run_[:, -1:]
    above = run_ > st["u"].double()[:, None] * total
    token = torch.where(t[:, 0] > 0, above.long().argmax(1), order[:, 0])
    logprob = torch.where(t[:, 0] > 0, (w.gather(1, token[:, None]) / total)[:, 0].log(), 0)
    return {"token": token.int(), "logprob": logprob.float()}


def run(st):
    case = st["case"]
    if not own:
        return {"linear": _linear_plain, "shared": _shared_plain, "sample": _sample_plain}[case["op"]](st)
    import ternary_weight_base_amd as tq
    if case["op"] == "linear":
        if "scratch" not in st:  # a server keeps one
            st["scratch"] = tq.linear_attn_scratch(st["total"], case["seqs"], case["q_heads"], case["kv_heads"], case["dim"])
        tq.tq_linear_attn(st["qkv"], st["decay"], st["cu"], st["from"], st["to"], st["states"], st["out"], scratch=st["scratch"])
        return {"out": st["out"], "states": st["states"]}
    if case["op"] == "shared":
        if "ws" not in st:
            st["ws"] = tq.kv_attn_shared_workspace(st["total"], case["seqs"], case["groups"], case["q_heads"], case["kv_heads"],
                                                   case["dim"], st["most_prefix"], st["most_own"])
        tq.tq_kv_attn_shared(st["q"], st["cu"], st["kv"], st["cu_seqs"], st["prefix"], st["table"], st["k"], st["v"], st["ks"],
                             st["vs"], st["out"], st["most_prefix"], st["most_own"], ws=st["ws"])
        return st["out"]
    if "ws" not in st:
        st["ws"] = tq.sample_workspace(case["rows"], case["vocab"])
    tq.tq_sample(st["logits"], st["u"], st["token"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                 min_p=st["min_p"], logprob=st["logprob"], ws=st["ws"])
    return {"token": st["token"], "logprob": st["logprob"]}


def work(case):
    size = {"f16": 2, "f32": 4}
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * size[case["dtype"]] + 24), "flops": 8 * case["rows"] * case["vocab"]}
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "linear":
        rows, seqs = sum(_rows(case)), case["seqs"]
        states = seqs * hkv * dim * dim * 4 * (1 if case["fresh"] else 2)
        decay = 4 * hkv * (rows if case["decay"] == "rows" else 1)
        return {"bytes": rows * ((hq + 2 * hkv) * dim * size[case["dtype"]] + 2 * hq * dim) + states + decay,
                "flops": rows * dim * dim * (3 * hkv + 2 * hq)}
    n, own_tokens, members, prefix = _sharing(case)
    group = [i for i, m in enumerate(members) for _ in range(m)]
    pairs = sum(x * prefix[group[s]] + sum(own_tokens[s] - x + 1 + i for i in range(x)) for s, x in enumerate(n))
    held = sum(prefix) + sum(own_tokens)
    return {"bytes": 2 * held * hkv * dim + 4 * sum(n) * hq * dim, "flops": 4 * pairs * hq * dim}


def _linear_exact(case, st):
    # token by token, all sequences side by side
    n = _rows(case)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    f8 = torch.float64
    cu = _starts(n)
    x = st["qkv"].to(f8).view(-1, hq + 2 * hkv, dim)
    a = st["decay"].to(f8).exp().expand(st["total"], hkv)
    states = st["states"].to(f8)
    s = torch.zeros((case["seqs"], hkv, dim, dim), dtype=f8, device="cuda")
    if not case["fresh"]:
        s = states[st["from"].long()].clone()
    out = torch.empty((st["total"], hq, dim), dtype=f8, device="cuda")
    for i in range(max(n)):
        live = [j for j in range(case["seqs"]) if i < n[j]]
        at = _device([cu[j] + i for j in live], torch.long)
        y, live = x[at], _device(live, torch.long)
        s[live] = s[live] * a[at][:, :, None, None] + y[:, hq:hq + hkv, :, None] * y[:, hq + hkv:, None, :]
        o = (y[:, :hq].reshape(-1, hkv, hq // hkv, dim, 1) * s[live][:, :, None]).sum(3)
        out[at] = o.reshape(-1, hq, dim) / math.sqrt(dim)
    states[st["to"].long()] = s
    return {"out": out, "states": states}


def _shared_exact(case, st):
    n, own_tokens, members, prefix = _sharing(case)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    f8, cu = torch.float64, _starts(n)
    group = [i for i, m in enumerate(members) for _ in range(m)]
    out = torch.empty((st["total"], hq, dim), dtype=f8, device="cuda")
    for s, (x, t) in enumerate(zip(n, own_tokens)):
        t += prefix[group[s]]
        ids = st["table"][s, :-(-t // PAGE)].long()
        hide = torch.arange(t, device="cuda").unsqueeze(0) > torch.arange(t - x, t, device="cuda").unsqueeze(1)
        for h in range(hkv):
            k = ((st["k"][ids, h].to(f8) - 127.5) * st["ks"][ids, h].to(f8)[:, None, None]).reshape(-1, dim)[:t].t().contiguous()
            v = (st["v"][ids, h].to(f8) - 127.5) * st["vs"][ids, h].to(f8)[:, None, None]
            v = v.transpose(1, 2).reshape(-1, dim)[:t].contiguous()
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                z = (st["q"][cu[s]:cu[s] + x, g].to(f8) @ k) / math.sqrt(dim)
                out[cu[s]:cu[s] + x, g] = torch.softmax(z.masked_fill(hide, -math.inf), 1) @ v
    return out


def _sample_exact(case, st):
    # row by row on the host: the kept tokens by their rank, then one running sum in index order
    rows = case["rows"]
    host = {k: None if st[k] is None else st[k].cpu().numpy().astype(np.float64) for k in
            ("logits", "u", "temperature", "top_k", "top_p", "min_p")}
    token, logprob = [], []
    for r in range(rows):
        x, t = host["logits"][r], host["temperature"][r]
        if t <= 0:
            token.append(int(x.argmax()))
            logprob.append(0.0)
            continue
        w = np.exp((x - x.max()) / t)
        rank = np.lexsort((np.arange(x.size), -x))
        k = 0 if host["top_k"] is None else int(host["top_k"][r])
        if k > 0:
            rank = rank[:k]
        if host["top_p"] is not None and host["top_p"][r] < 1:
            c = np.cumsum(w[rank])
            rank = rank[:int(np.searchsorted(c, host["top_p"][r] * c[-1], side="left")) + 1]
        if host["min_p"] is not None:
            rank = rank[w[rank] >= host["min_p"][r]]
        kept = np.sort(rank)
        c = np.cumsum(w[kept])
        i = kept[min(int(np.searchsorted(c, host["u"][r] * c[-1], side="right")), kept.size - 1)]
        token.append(int(i))
        logprob.append(math.log(w[i] / c[-1]))
    return {"token": _device(token), "logprob": _device(logprob, torch.float64)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _linear_exact, "shared": _shared_exact, "sample": _sample_exact}[case["op"]](case, st)
