"""The recurrence of linear attention token by token in float64 (elementary
torch operations, on any device), and how far fp32 states and fp16 outputs
may be from it."""
import math

import torch

F8 = torch.float64
U = 2.0 ** -24  # half an fp32 step
FEW = 16        # rows a sequence, on average, up to which the recurrence runs row by row


def linear(qkv, log_decay, cu, start, to, states, scale, hq, hkv, dim):
    """-> out [rows][hq][dim], its magnitude (sums of absolute values), {state
    index: (state, magnitude)}, log2 decays a sequence and head summed."""
    rows, dev = qkv.shape[0], qkv.device
    x = qkv.to(F8).reshape(rows, hq + 2 * hkv, dim)
    g = (log_decay.to(F8) / math.log(2)).clamp(max=0).expand(rows, hkv)
    out = torch.full((rows, hq, dim), math.nan, dtype=F8, device=dev)
    mag = torch.full_like(out, math.nan)
    left, fall = {}, {}
    for s in range(len(start)):
        a, b = cu[s], cu[s + 1]
        if b <= a:
            continue
        S = torch.zeros((hkv, dim, dim), dtype=F8, device=dev)
        if 0 <= start[s] < states.shape[0]:
            S = states[start[s]].to(F8).clone()
        M = S.abs()
        for r in range(a, b):
            q, k, v = x[r, :hq].reshape(hkv, hq // hkv, dim), x[r, hq:hq + hkv], x[r, hq + hkv:]
            d = torch.exp2(g[r])[:, None, None]
            S = torch.where(d > 0, d * S, 0) + k[:, :, None] * v[:, None, :]
            M = torch.where(d > 0, d * M, 0) + k.abs()[:, :, None] * v.abs()[:, None, :]
            out[r] = scale * (q[..., None] * S[:, None]).sum(2).reshape(hq, dim)
            mag[r] = abs(scale) * (q.abs()[..., None] * M[:, None]).sum(2).reshape(hq, dim)
        fall[s] = g[a:b].clamp(min=-2000).sum(0).abs()[:, None, None]
        if 0 <= to[s] < states.shape[0]:
            left[to[s]] = (S, M, s)
    return out, mag, left, fall


def chunked(cu):
    return cu[-1] > FEW * (len(cu) - 1)


def state_tolerance(M, n, fall, chunks_form):
    """Errors of a state's element relative to M, the sum of its terms' absolute
    values (terms: decayed products of a key and a value, the start).
    Row by row: a decay is an exp2 (one fp32 step, 2 U) of a rounded argument
    (U of it), its product and the sum one rounding each: n (5 U) and U times the
    log2 decays' sum (times ln 2 < 1).
    In chunks: a weight is an exp2 of a rounded sum and a product (4 U and the
    sums' U); two fp16 terms a factor, both cut off, leave 2^-20 of it, and the
    product of the second terms is 2^-20 (48 U for both factors and that); 3 x 128
    terms are added in fp32 (384 U), each chunk's state with two roundings and a
    decay of 2 U: 4 U a chunk.  fp16's least step, half of 2^-24 under a largest
    element of at least 2^13, is 2^-38 of a tile's largest key times a value
    (and the reverse), in up to 64 terms a tile: 2^-30 of the largest M."""
    if not chunks_form:
        return (5 * n + fall + 4) * U * M
    return (440 + 4 * math.ceil(n / 128) + 2 * fall) * U * M + 2.0 ** -30 * M.amax((1, 2), keepdim=True)


def out_tolerance(ref, mag, most, n, fall, dim, chunks_form):
    """Row by row: the state's error, the query's scaling and dim products and
    sums in fp32, then fp16 (half a step, 2^-11, or half of the least one).
    In chunks: of the factors of a term, the state (of a term with it) or the fp32
    value (of the others) is rounded once to fp16 (2^-11); query, key and weight
    have two terms and lose 2^-20 each, 2^-20 more for a product of second
    terms (64 U), dim products and sums of a score and up to 500 of an output
    are in fp32, three terms each.  Small parts of a tile as for
    states: 2^-30 of the largest magnitude `most` of the sequence and head."""
    t = 2.0 ** -11 * ref.abs() + 2.0 ** -25
    if not chunks_form:
        return t + (5 * n + fall + dim + 8) * U * mag
    return t + (2.0 ** -11 + (3 * dim + 64 + 2 * 500 + 2 * fall) * U) * mag + 2.0 ** -30 * most


def check(got_out, got_states, qkv, log_decay, cu, start, to, states, scale, hq, hkv, dim):
    """Asserts outputs and states; rows outside the sequences and states that no
    one writes must be as they were (`states`: before the call; rows: NaN)."""
    out, mag, left, fall = linear(qkv, log_decay, cu, start, to, states, scale, hq, hkv, dim)
    form = chunked(cu)
    for s in range(len(start)):
        a, b = cu[s], cu[s + 1]
        if b <= a:
            continue
        f = fall[s].reshape(1, hkv, 1, 1)
        sh = (b - a, hkv, hq // hkv, dim)
        ref, m = out[a:b].reshape(sh), mag[a:b].reshape(sh)
        tol = out_tolerance(ref, m, m.amax((0, 2, 3), keepdim=True), b - a, f, dim, form)
        got = got_out[a:b].to(F8).reshape(sh)
        err = (got - ref).abs()
        # from 65520 on fp16 rounds to infinity
        err = torch.where(torch.isinf(got) & (got * ref > 0) & (ref.abs() + tol >= 65520), 0, err)
        assert bool((err <= tol).all()), f"out of sequence {s}: {float((err / tol).max())} of the tolerance"
    for i in range(states.shape[0]):
        if i not in left:
            assert torch.equal(got_states[i].view(torch.int32), states[i].view(torch.int32)), f"state {i} changed"
            continue
        S, M, s = left[i]
        err = (got_states[i].to(F8) - S).abs()
        tol = state_tolerance(M, cu[s + 1] - cu[s], fall[s], form)
        assert bool((err <= tol).all()), f"state {i}: {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"
    assert bool(torch.isnan(got_out[cu[-1]:]).all()), "rows behind the last sequence changed"
