"""Plain 64-bit implementations (torch, CPU) of the products whose second
matrix is chosen row by row, and the error bounds their tests use."""
import math

import torch

INF = math.inf
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest subnormal


def route(logits, k, bias=None, score="softmax", groups=1, keep_groups=1, group_top=1, normalize=False, scale=1.0):
    """(weight, index, s) one row and one choice at a time."""
    l = logits.double()
    T, E = l.shape
    weight = torch.zeros(T, k, dtype=torch.float64)
    index = torch.full((T, k), -1, dtype=torch.int32)
    scores = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        row = l[t].tolist()
        if score == "sigmoid":
            s = [1.0 / (1.0 + math.exp(-x)) if x > -700 else (x if x != x else 0.0) for x in row]
        else:
            known = [x for x in row if x == x]
            m = max(known) if known else 0.0
            if m == -INF:
                m = 0.0
            e = [x if x != x else INF - INF if x == INF else math.exp(x - m) if x - m > -745 else 0.0 for x in row]
            total = sum(e)
            s = [x / total if total != 0 else 0.0 for x in e]
        scores[t] = torch.tensor(s, dtype=torch.float64)
        b = [0.0] * E if bias is None else bias.double().tolist()
        there = [row[e] != -INF and b[e] != -INF for e in range(E)]
        c = [s[e] + b[e] for e in range(E)]

        def rank(x):       # NaN first
            return (1, 0.0) if x != x else (0, x)
        allowed = set(e for e in range(E) if there[e])
        if groups > 1:
            per = E // groups
            value = []
            for q in range(groups):
                mine = sorted((rank(c[e]) for e in range(q * per, (q + 1) * per) if there[e]), reverse=True)
                if not mine:
                    value.append((-1, 0.0))
                elif mine[0][0] == 1:
                    value.append((1, 0.0))
                else:
                    value.append((0, sum(x for _, x in mine[:group_top])))
            kept = sorted(range(groups), key=lambda q: (-value[q][0], -value[q][1], q))[:keep_groups]
            allowed = set(e for e in allowed if e // per in kept)
        key = c if bias is not None else row
        picks = sorted(allowed, key=lambda e: (-rank(key[e])[0], -rank(key[e])[1], e))[:k]
        w = [s[e] for e in picks]
        if normalize:
            if score == "softmax" and picks:       # the row's sum cancels: take it over the chosen alone
                known = [row[e] for e in picks if row[e] == row[e]]
                m = max(known) if known else 0.0
                w = [x if x != x else INF - INF if x == INF else math.exp(x - m) if x - m > -745 else 0.0
                     for x in (row[e] for e in picks)]
            total = sum(w)
            w = [x / total if total != 0 else 0.0 for x in w]
        for j, e in enumerate(picks):
            index[t, j] = e
            weight[t, j] = w[j] * scale
    return weight, index, scores


def route_weight_of(l, index, score, normalize, scale):
    """weight as a differentiable 64-bit function of the logits, the choice given."""
    ok = index >= 0
    at = index.clamp_min(0).long()
    if score == "sigmoid":
        s = torch.sigmoid(l)
        w = torch.where(ok, s.gather(1, at), torch.zeros((), dtype=l.dtype))
        if normalize:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    elif normalize:
        x = torch.where(ok, l.gather(1, at), torch.full((), -INF, dtype=l.dtype))
        x = torch.where(ok.any(1, keepdim=True), x, torch.zeros((), dtype=l.dtype))
        w = torch.where(ok, torch.softmax(x, 1), torch.zeros((), dtype=l.dtype))
    else:
        alive = torch.where((l > -INF).any(1, keepdim=True), l, torch.zeros((), dtype=l.dtype))
        w = torch.where(ok, torch.softmax(alive, 1).gather(1, at), torch.zeros((), dtype=l.dtype))
    return w * scale


def route_grad(logits, index, dweight, score, normalize, scale):
    """The formula's gradient, by autograd in 64 bits."""
    l = logits.double().clone().requires_grad_(True)
    w = route_weight_of(l, index, score, normalize, scale)
    (w * torch.where(index >= 0, dweight.double(), torch.zeros((), dtype=torch.float64))).sum().backward()
    return torch.nan_to_num(l.grad, nan=0.0)


def expert_map(index, experts):
    flat = index.reshape(-1).tolist()
    members = [[] for _ in range(experts)]
    for s, x in enumerate(flat):
        if 0 <= x < experts:
            members[x].append(s)
    order, offsets = [], [0]
    for mine in members:
        order += mine
        offsets.append(len(order))
    position = [-1] * len(flat)
    for p, s in enumerate(order):
        position[s] = p
    order += [-1] * (len(flat) - len(order))
    i32 = torch.int32
    return torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32), torch.tensor(position, dtype=i32).reshape(index.shape)


def rows_of(X, order, per_row):
    """The rows of X that the places of `order` name, zeros for -1."""
    out = torch.zeros(len(order), X.shape[1], dtype=torch.float64)
    for p, s in enumerate(order.tolist()):
        if s >= 0 and s // per_row < X.shape[0]:
            out[p] = X[s // per_row].double()
    return out


def close(got, want, bound, what=""):
    """|got - want| <= bound per element, NaN and infinities equal."""
    got, want = got.double().cpu(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= bound))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at "
                           f"{torch.nonzero(bad)[0].tolist()}: got {got[bad][0]!r} want {want[bad][0]!r} "
                           f"bound {torch.as_tensor(bound).expand(bad.shape)[bad][0]!r}")


def product_bound(want, magnitude, terms, dtype):
    """Bound for a sum of `terms` products rounded once to dtype.

    Each of at most `terms` products and additions in binary32 is off by at
    most a whole step (2^-23; half a step where the matrix cores round to
    nearest) of a partial sum that is no larger than `magnitude`, the sum of the products'
    magnitudes; the result is rounded by half a step of its type.
    """
    err = 2.0 * terms * 2.0 ** -23 * magnitude
    return err + STEP[dtype] * (want.abs() + err) + TINY[dtype]
