"""The operators between the projections of a decoder layer, and the cases they are measured on.

  append  tq_kv_append: rotate queries and keys by position, append keys and values to the paged 8-bit cache
  attn    tq_kv_attn: attention of the new rows over that cache (causal; optional sliding window with sink tokens)
  norm    tq_residual_norm: norm after a block, gate, residual scale, residual add, norm before the next block

The cache holds a byte b as the value (b - 127.5) * s with one power-of-two scale s for each page of 64 tokens and
KV head: K as [pages][heads][64][dim], V as [pages][heads][dim][64].
"""
import math
import random

import torch

own = False

PAGE = 64
# (query heads, KV heads, head dim); the first is this repository's 27B-shaped layer (QKV 5120 -> 10240)
HEADS = ((64, 8, 128), (32, 8, 128), (40, 8, 128), (16, 16, 64), (24, 4, 64))
HIDDEN = 5120


def listed():
    a, b, c = HEADS[0], HEADS[1], HEADS[3]

    def heads(h):
        return {"q_heads": h[0], "kv_heads": h[1], "dim": h[2]}

    return [
        # one user's next token: the whole call is latency
        {"name": "append_1", "op": "append", **heads(a), "seqs": 1, "rows": 1, "kv": 1000, "ragged": False, "dtype": "f32",
         "rot": 128, "pairs": False},
        # a server's step: 64 sequences of different lengths, one token each, fp16 projections, interleaved pairs
        {"name": "append_64", "op": "append", **heads(b), "seqs": 64, "rows": 1, "kv": 2000, "ragged": True, "dtype": "f16",
         "rot": 128, "pairs": True},
        # prompts of three users at once, none a multiple of a page, on contexts that end inside a page
        {"name": "append_prompt", "op": "append", **heads(a), "seqs": 3, "rows": 2051, "kv": 2500, "ragged": True, "dtype": "f32",
         "rot": 128, "pairs": False},
        # one user, a short chat so far: latency
        {"name": "attn_1_short", "op": "attn", **heads(a), "seqs": 1, "rows": 1, "kv": 517, "ragged": False, "window": 0, "sinks": 0},
        # one user, a long document: one token over 128 K of cache
        {"name": "attn_1_long", "op": "attn", **heads(a), "seqs": 1, "rows": 1, "kv": 131001, "ragged": False, "window": 0, "sinks": 0},
        # a server's step over ragged contexts
        {"name": "attn_64", "op": "attn", **heads(a), "seqs": 64, "rows": 1, "kv": 8190, "ragged": True, "window": 0, "sinks": 0},
        # four drafted tokens a sequence to verify
        {"name": "attn_drafts", "op": "attn", **heads(a), "seqs": 8, "rows": 4, "kv": 6001, "ragged": True, "window": 0, "sinks": 0},
        # sliding window with sink tokens, one KV head a query head
        {"name": "attn_window", "op": "attn", **heads(c), "seqs": 16, "rows": 1, "kv": 20011, "ragged": True, "window": 4000, "sinks": 4},
        # a prompt of 4096 tokens
        {"name": "attn_prompt", "op": "attn", **heads(a), "seqs": 1, "rows": 4096, "kv": 4096, "ragged": False, "window": 0, "sinks": 0},
        # pieces of two prompts on earlier context, with window and sinks, five query heads a KV head
        {"name": "attn_chunks", "op": "attn", **heads(HEADS[2]), "seqs": 2, "rows": 1025, "kv": 9001, "ragged": True, "window": 2047,
         "sinks": 64},
        # one token between two blocks: latency
        {"name": "norm_1", "op": "norm", "rows": 1, "hidden": HIDDEN, "y": "f32", "res": "f32", "x": "f16", "post": True, "gate": "vector"},
        # a prompt's rows between two blocks, quantised for the prefill GEMM
        {"name": "norm_prompt", "op": "norm", "rows": 2048, "hidden": HIDDEN, "y": "f32", "res": "f32", "x": "i8", "post": True,
         "gate": "rows"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("append", "attn", "attn", "attn", "norm"))
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 2048), "hidden": _log(rng, 64, 5120), "y": rng.choice(("f16", "f32")),
                "res": rng.choice(("f16", "f32")), "x": rng.choice(("f16", "f32", "i8")), "post": rng.random() < 0.7,
                "gate": rng.choice(("none", "vector", "rows"))}
    h = rng.choice(HEADS)
    c = {"op": op, "q_heads": h[0], "kv_heads": h[1], "dim": h[2]}
    many = rng.random() < 0.4
    if many:
        c |= {"seqs": rng.randint(1, 3), "rows": _log(rng, 17, 2000)}
        c["kv"] = c["rows"] + _log(rng, 1, 4000)
    else:
        c |= {"seqs": _log(rng, 1, 64), "rows": rng.choice((1, 1, 2, 3, 4))}
        c["kv"] = c["rows"] + _log(rng, 1, 2000 if op == "append" else 8000)
    c["ragged"] = rng.random() < 0.7
    if op == "append":
        c |= {"dtype": rng.choice(("f16", "f32")), "rot": rng.choice((h[2], h[2] // 2)), "pairs": rng.random() < 0.5}
    else:
        w = rng.random() < 0.4
        c |= {"window": _log(rng, 1, 4000) if w else 0, "sinks": rng.choice((0, 1, 4, 70)) if w else 0}
    while c["seqs"] > 1 and (work(c)["flops"] > 2.7e11 or work(c)["bytes"] > 6.5e8):
        c["seqs"] -= 1
    return c


DTYPES = {"f16": torch.float16, "f32": torch.float32, "i8": torch.int8}


def _lens(case):
    """(new rows, tokens in the cache after them) of each sequence: spread below the case's largest where it is ragged."""
    r = random.Random("%(seqs)d %(rows)d %(kv)d" % case)
    n, kv = [], []
    for s in range(case["seqs"]):
        big = s == 0 or not case["ragged"]
        n.append(case["rows"] if big else r.randint((case["rows"] + 1) // 2, case["rows"]))
        kv.append(case["kv"] if big else max(n[-1], r.randint(case["kv"] // 4, case["kv"])))
    return n, kv


def _cache(case, g):
    n, kv = _lens(case)
    heads, dim = case["kv_heads"], case["dim"]
    width = -(-max(kv) // PAGE)
    used = [-(-x // PAGE) for x in kv]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(n), width), -1, dtype=torch.int32, device="cuda")  # no page where a sequence has ended
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u

    def codes(*shape):
        # normal values, their largest using the upper half of the bytes' range, as a power-of-two scale leaves it
        spread = 28 * (0.5 + 0.5 * torch.rand((pages, heads, 1, 1), generator=g, device="cuda"))
        x = torch.randn(shape, generator=g, device="cuda").mul_(spread).add_(128).floor_().clamp_(0, 255)
        return x.to(torch.uint8)

    def scales():
        e = torch.randint(-6, -3, (pages, heads), generator=g, device="cuda").int()
        return ((e + 127) << 23).view(torch.float32)  # powers of two

    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return {"cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "kv": torch.tensor(kv, dtype=torch.int32, device="cuda"),
            "table": table, "total": cu[-1], "most_rows": max(n), "most_kv": max(kv),
            "k": codes(pages, heads, PAGE, dim), "v": codes(pages, heads, dim, PAGE), "ks": scales(), "vs": scales()}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "norm":
        m, h = case["rows"], case["hidden"]
        q = case["x"] == "i8"
        st = {"case": case, "y": (3 * torch.randn((m, h), generator=g, device="cuda")).to(DTYPES[case["y"]]),
              "res": (2 * torch.randn((m, h), generator=g, device="cuda")).to(DTYPES[case["res"]]),
              "pre": 1 + 0.1 * torch.randn(h, generator=g, device="cuda"), "post": None, "gate": None,
              "scale": 0.7, "eps": 1e-6}
        if case["post"]:
            st["post"] = 1 + 0.1 * torch.randn(h, generator=g, device="cuda")
        if case["gate"] != "none":
            shape = (h,) if case["gate"] == "vector" else (m, h)
            st["gate"] = torch.tanh(torch.randn(shape, generator=g, device="cuda")).to(DTYPES[case["y"]])
        st["res_out"] = torch.empty_like(st["res"])
        st["x"] = torch.empty((m, h), dtype=DTYPES[case["x"]], device="cuda")
        st["a"] = torch.empty(m, device="cuda") if q else None
        return st
    st = {"case": case, **_cache(case, g)}
    rows, hq, hkv, dim = st["total"], case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        st["qkv"] = (1.5 * torch.randn((rows, (hq + 2 * hkv) * dim), generator=g, device="cuda")).to(DTYPES[case["dtype"]])
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(st["most_kv"], device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / case["rot"])
        st["rope"] = torch.stack((angle.cos(), angle.sin()), 1).float()
        st["q"] = torch.zeros((rows, hq, dim), dtype=torch.float16, device="cuda")
        # the pages that receive rows: where the updated cache is read
        page = _places(st)[0]
        st["pages"] = torch.unique(page).int()
        st["values"] = torch.empty((2, st["pages"].numel(), hkv, PAGE, dim), dtype=torch.float16, device="cuda")
    else:
        st["q"] = (2 * torch.randn((rows, hq, dim), generator=g, device="cuda")).half()
        st["out"] = torch.zeros_like(st["q"])
    return st


def _places(st):
    """(page, slot in it, position, sequence) of each row."""
    r = torch.arange(st["total"], device="cuda")
    seq = (r[:, None] >= st["cu"][None, 1:]).sum(1)
    pos = st["kv"].long()[seq] - (st["cu"].long()[seq + 1] - r)
    return st["table"].long()[seq, pos // PAGE], pos % PAGE, pos, seq


def _store(codes, scale, x, pages, page, slot, token_axis):
    """Appends the rows x [rows][heads][dim] to codes and scale, in place."""
    heads = x.shape[1]
    most = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, heads), x.abs().amax(-1), "amax")[pages]
    first = torch.full((codes.shape[0],), PAGE, device="cuda").scatter_reduce(0, page, slot, "amin")[pages]
    e = torch.frexp(most).exponent.long() - 7  # the least e with most < 128 * 2^e
    need = torch.where(most > 0, ((e.clamp(min=-126) + 127) << 23).int().view(torch.float32), 0)
    old = torch.where((first == 0)[:, None], 0, scale[pages])
    new = torch.maximum(old, need)
    grow = torch.where(old > 0, (new.view(torch.int32) >> 23) - (old.view(torch.int32) >> 23), 0).clamp(max=8)
    sub = codes[pages].int() - 128
    shape = [1, 1, 1, 1]
    shape[token_axis] = PAGE
    before = torch.arange(PAGE, device="cuda").view(shape) < first[:, None, None, None]
    codes[pages] = (torch.where(before, sub >> grow[:, :, None, None], sub) + 128).to(torch.uint8)
    scale[pages] = new
    s = scale[page].double()[:, :, None]
    c = torch.where(s > 0, torch.floor(x.double() / torch.where(s > 0, s, 1)), 0).clamp(-128, 127) + 128
    if token_axis == 2:
        codes[page, :, slot] = c.to(torch.uint8)
    else:
        codes[page, :, :, slot] = c.to(torch.uint8)


def _append_plain(st):
    case = st["case"]
    hq, hkv, dim, rot = case["q_heads"], case["kv_heads"], case["dim"], case["rot"]
    page, slot, pos, _ = _places(st)
    x = st["qkv"].view(-1, hq + 2 * hkv, dim)
    qk, t = x[:, :hq + hkv].double(), st["rope"].double()[pos]
    c, s = t[:, None, 0], t[:, None, 1]
    if case["pairs"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    qk = torch.cat((turned, qk[..., rot:]), -1).float()
    pages = st["pages"].long()
    _store(st["k"], st["ks"], qk[:, hq:], pages, page, slot, 2)
    _store(st["v"], st["vs"], x[:, hq + hkv:].float(), pages, page, slot, 3)
    k = (st["k"][pages].float() - 127.5) * st["ks"][pages][:, :, None, None]
    v = (st["v"][pages].float() - 127.5) * st["vs"][pages][:, :, None, None]
    return {"q": qk[:, :hq].half(), "values": torch.stack((k, v.transpose(2, 3))).half(), "k_scale": st["ks"], "v_scale": st["vs"]}


def _attn_plain(st):
    case = st["case"]
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    seqs, n, width, group = case["seqs"], st["most_rows"], st["table"].shape[1], hq // hkv
    cu, kv, table = st["cu"].long(), st["kv"].long(), st["table"].long().clamp(min=0)
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=st["total"] - 1)
    q = st["q"][row].float().view(seqs, n, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * n, dim)
    k = (st["k"][table].float() - 127.5) * st["ks"][table][..., None, None]
    k = k.transpose(1, 2).reshape(seqs, hkv, width * PAGE, dim)
    score = torch.matmul(q, k.transpose(2, 3)).view(seqs, hkv, group, n, width * PAGE) * dim ** -0.5
    del k
    pos = (kv - count)[:, None, None] + i[None, :, None]
    j = torch.arange(width * PAGE, device="cuda")
    seen = j <= pos
    if case["window"]:
        seen &= (j > pos - case["window"]) | (j < case["sinks"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1)
    v = (st["v"][table].float() - 127.5) * st["vs"][table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(seqs, hkv, width * PAGE, dim)
    o = torch.matmul(p.view(seqs, hkv, group * n, width * PAGE), v).view(seqs, hkv, group, n, dim)
    o = torch.where(total > 0, 1 / total, 0)[..., None] * o
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, n, hq, dim).half()
    return o[i < count[:, None]]  # the rows in order


def _norm_plain(st):
    u, r = st["y"].double(), st["res"].double()
    if st["post"] is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + st["eps"]) * st["post"].double()
    if st["gate"] is not None:
        u = u * st["gate"].double()
    r = (r + st["scale"] * u).float().to(st["res"].dtype)
    w = r.double()
    x = (w * torch.rsqrt(w.square().mean(-1, keepdim=True) + st["eps"]) * st["pre"].double()).float()
    if st["a"] is None:
        return {"res": r, "x": x.to(st["x"].dtype)}
    most = x.abs().amax(-1, keepdim=True)
    q = torch.round(x * (127 / most)).clamp(-127, 127)
    return {"res": r, "x": q * (most / 127), "a": (most / 127)[:, 0]}


def run(st):
    case = st["case"]
    if not own:
        return {"append": _append_plain, "attn": _attn_plain, "norm": _norm_plain}[case["op"]](st)
    import ternary_weight_base_amd as tq
    if case["op"] == "append":
        tq.tq_kv_append(st["qkv"], st["rope"], st["cu"], st["kv"], st["table"], st["k"], st["v"], st["ks"], st["vs"], st["q"],
                        rope_mode=tq.TQ_ROPE_PAIRS if case["pairs"] else tq.TQ_ROPE_HALVES)
        tq.tq_debug_kv_read(st["pages"], st["k"], st["v"], st["ks"], st["vs"], st["values"])
        return {"q": st["q"], "values": st["values"], "k_scale": st["ks"], "v_scale": st["vs"]}
    if case["op"] == "attn":
        if "ws" not in st:  # a server keeps one workspace
            st["ws"] = tq.kv_attn_workspace(st["total"], case["seqs"], case["q_heads"], case["kv_heads"], case["dim"], st["most_kv"])
        tq.tq_kv_attn(st["q"], st["cu"], st["kv"], st["table"], st["k"], st["v"], st["ks"], st["vs"], st["out"], st["most_kv"],
                      window=case["window"], sinks=case["sinks"], ws=st["ws"])
        return st["out"]
    if st["a"] is None:
        tq.tq_residual_norm(st["y"], st["res"], st["res_out"], st["pre"], x=st["x"], post_w=st["post"], gate=st["gate"],
                            res_scale=st["scale"], eps=st["eps"])
        return {"res": st["res_out"], "x": st["x"]}
    tq.tq_residual_norm(st["y"], st["res"], st["res_out"], st["pre"], q=st["x"], a_scale=st["a"], post_w=st["post"], gate=st["gate"],
                        res_scale=st["scale"], eps=st["eps"])
    return {"res": st["res_out"], "x": st["x"] * st["a"][:, None], "a": st["a"]}


def _seen(case, p):
    """How many keys a row at position p sees."""
    if not case["window"]:
        return p + 1
    first = max(0, p - case["window"] + 1)
    return p + 1 - first + min(case["sinks"], first)


def work(case):
    size = {"f16": 2, "f32": 4, "i8": 1}
    if case["op"] == "norm":
        m, h = case["rows"], case["hidden"]
        gate = {"none": 0, "vector": h, "rows": m * h}[case["gate"]] * size[case["y"]]
        out = m * h * (5 if case["x"] == "i8" else size[case["x"]])  # int8 and the values it stands for
        return {"bytes": m * h * (size[case["y"]] + 2 * size[case["res"]]) + gate + out + 4 * h * (1 + case["post"]), "flops": 12 * m * h}
    n, kv = _lens(case)
    rows, hq, hkv, dim = sum(n), case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        pages = sum(-(-t // PAGE) - (t - x) // PAGE for x, t in zip(n, kv))
        read = rows * ((hq + 2 * hkv) * dim * size[case["dtype"]] + 4 * case["rot"])
        # the touched pages read back: bytes in, values out
        back = 2 * pages * hkv * PAGE * dim * 3
        return {"bytes": read + rows * (2 * hq + 2 * hkv) * dim + back, "flops": 6 * rows * (hq + hkv) * case["rot"] // 2}
    pairs = sum(sum(_seen(case, t - x + i) for i in range(x)) for x, t in zip(n, kv))
    held = 0  # tokens that some row of the sequence sees
    for x, t in zip(n, kv):
        first = max(0, t - x - case["window"] + 1) if case["window"] else 0
        held += t - first + min(case["sinks"], first)
    return {"bytes": 2 * held * hkv * dim + 4 * rows * hq * dim, "flops": 4 * pairs * hq * dim}


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        y, r = st["y"].to(f8), st["res"].to(f8)
        if st["post"] is not None:
            y = y / (y.pow(2).sum(1) / y.shape[1] + st["eps"]).sqrt().unsqueeze(1) * st["post"].to(f8)
        r = r + (y if st["gate"] is None else y * st["gate"].to(f8)) * st["scale"]
        stored = r.float().to(st["res"].dtype).to(f8)  # the next block's norm is of the stored residual
        x = stored / (stored.pow(2).sum(1) / r.shape[1] + st["eps"]).sqrt().unsqueeze(1) * st["pre"].to(f8)
        if st["a"] is None:
            return {"res": r, "x": x}
        return {"res": r, "x": None, "a": x.abs().max(1).values / 127}
    n, kv = _lens(case)
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    group = hq // hkv
    if case["op"] == "attn":
        out = torch.empty((st["total"], hq, dim), dtype=f8, device="cuda")
        at = 0
        for s, (x, t) in enumerate(zip(n, kv)):
            ids = st["table"][s, :-(-t // PAGE)].long()
            pos = torch.arange(t - x, t, device="cuda").unsqueeze(1)
            key = torch.arange(t, device="cuda").unsqueeze(0)
            hide = key > pos
            if case["window"]:
                hide = hide | ((pos - key >= case["window"]) & (key >= case["sinks"]))
            for h in range(hkv):
                k = ((st["k"][ids, h].to(f8) - 127.5) * st["ks"][ids, h].to(f8)[:, None, None]).reshape(-1, dim)[:t]
                v = (st["v"][ids, h].to(f8) - 127.5) * st["vs"][ids, h].to(f8)[:, None, None]
                v = v.transpose(1, 2).reshape(-1, dim)[:t].contiguous()
                for g in range(group):
                    z = (st["q"][at:at + x, h * group + g].to(f8) @ k.t().contiguous()) / math.sqrt(dim)
                    out[at:at + x, h * group + g] = torch.softmax(z.masked_fill(hide, -math.inf), 1) @ v
            at += x
        return out
    # append: sequence by sequence, page by page
    rows = st["qkv"].to(f8).view(-1, hq + 2 * hkv, dim)
    rot = case["rot"]
    q = torch.empty((st["total"], hq, dim), dtype=f8, device="cuda")
    where = {int(p): i for i, p in enumerate(st["pages"].tolist())}
    kc, vc = st["k"].to(torch.int64) - 128, st["v"].transpose(2, 3).to(torch.int64) - 128
    ks, vs = st["ks"].clone(), st["vs"].clone()
    values = torch.empty(st["values"].shape, dtype=f8, device="cuda")
    at = 0
    for s, (x, t) in enumerate(zip(n, kv)):
        r = rows[at:at + x]
        turn = torch.complex(st["rope"][t - x:t, 0].to(f8), st["rope"][t - x:t, 1].to(f8)).unsqueeze(1)
        z = r[:, :hq + hkv].clone()
        if case["pairs"]:
            c = torch.complex(z[..., 0:rot:2].contiguous(), z[..., 1:rot:2].contiguous()) * turn
            z[..., 0:rot:2], z[..., 1:rot:2] = c.real, c.imag
        else:
            c = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous()) * turn
            z[..., :rot // 2], z[..., rot // 2:rot] = c.real, c.imag
        q[at:at + x] = z[:, :hq]
        done = 0
        while done < x:
            pos = t - x + done
            m = min(x - done, PAGE - pos % PAGE)
            page, a = int(st["table"][s, pos // PAGE]), pos % PAGE
            # keys are rounded to fp32 before they are cut into steps
            for new, c, sc in ((z[done:done + m, hq:].float().to(f8), kc, ks), (r[done:done + m, hq + hkv:], vc, vs)):
                most = new.abs().amax((0, 2)).tolist()
                for h in range(hkv):
                    before = float(sc[page, h]) if a else 0.0
                    need = 2.0 ** max(-126, math.frexp(most[h])[1] - 7) if most[h] else 0.0
                    now = max(before, need)
                    if before and now > before:
                        c[page, h, :a] = torch.div(c[page, h, :a], int(min(256, now / before)), rounding_mode="floor")
                    c[page, h, a:a + m] = torch.floor(new[:, h] / now).long() if now else 0
                    sc[page, h] = now
            i = where[page]
            values[0, i] = (kc[page] + 0.5) * ks[page].to(f8)[:, None, None]
            values[1, i] = (vc[page] + 0.5) * vs[page].to(f8)[:, None, None]
            done += m
        at += x
    return {"q": q, "values": values, "k_scale": ks.to(f8), "v_scale": vs.to(f8)}
