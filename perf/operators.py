"""Cases of the operators whose weight matrix is chosen row by row.

Routing of tokens to experts and its slot map, the experts' products, the
weighted sum of their results, and low-rank adapters of many requests beside a
shared projection.  `listed` and `draw` say what is run, `prepare` makes the
tensors a program holds before the call, `run` makes one pass: in plain torch
operations, or (`own`) through dense_fp32_gemm_amd.binding.  `exact` computes
the same outputs from the definitions in binary64.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _route(name, T, E, k, dtype, score, normalize, groups=1, keep=1, top=1, bias=False, scale=1.0, pad=0, grad=False):
    return dict(name=name, op="route", T=T, E=E, k=k, dtype=dtype, score=score, normalize=normalize, groups=groups,
                keep=keep, top=top, bias=bias, scale=scale, pad=pad, grad=grad)


def _experts(name, T, E, k, K, N, dtype, grad=False):
    return dict(name=name, op="experts", T=T, E=E, k=k, K=K, N=N, dtype=dtype, grad=grad)


def _combine(name, T, E, k, N, dtype, grad=False):
    return dict(name=name, op="combine", T=T, E=E, k=k, N=N, dtype=dtype, grad=grad)


def _adapters(name, T, K, N, R, n, requests, dtype):
    return dict(name=name, op="adapters", T=T, K=K, N=N, R=R, n=n, requests=requests, dtype=dtype)


def listed():
    return [
        # one decoding step of a small batch: latency
        _route("route_step", 16, 64, 4, "float32", "softmax", True),
        # a long prompt batch, sigmoid scores with a balance bias and groups; the last rows are padding (no expert available)
        _route("route_prompt", 8192, 256, 8, "float32", "sigmoid", True, 8, 4, 2, True, 2.5, pad=192),
        # a training batch with the gradient of the logits, odd number of rows
        _route("route_train", 16383, 128, 8, "bfloat16", "softmax", True, grad=True),
        # one decoding step: 32 slots, the weights of the chosen experts are what is read
        _experts("experts_step", 8, 32, 4, 2048, 1024, "bfloat16"),
        # a prompt batch over few experts in binary32
        _experts("experts_f32", 2048, 8, 2, 2048, 2048, "float32"),
        # a long prompt batch over many experts
        _experts("experts_prompt", 8192, 64, 8, 2048, 1024, "bfloat16"),
        # training: gradients of the rows and of the weights
        _experts("experts_train", 4096, 16, 4, 2048, 2048, "bfloat16", grad=True),
        # the same with sizes that fit no tile, in binary32
        _experts("experts_train_odd", 1025, 8, 2, 1000, 1023, "float32", grad=True),
        # the weighted sum of a decoding step
        _combine("combine_step", 16, 32, 4, 1000, "float32"),
        # the weighted sum of a training batch and its gradients
        _combine("combine_train", 8192, 64, 8, 2048, "bfloat16", grad=True),
        # one token of each of 32 requests, nearly every one with its own adapter
        _adapters("adapters_step", 32, 4096, 4096, 16, 64, 32, "bfloat16"),
        # prompts of a few requests together
        _adapters("adapters_prompt", 2050, 4096, 4096, 32, 8, 7, "float16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A row length: mostly a multiple of 64, else any number."""
    w = _spread(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def _drawn(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "adapters", "adapters"])
    dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _spread(rng, 2, 256 // groups) if groups > 1 else _spread(rng, 2, 256)
        keep = rng.randint(1, groups)
        k = min(rng.randint(1, 8), E // groups * keep)
        T = _spread(rng, 1, 16384)
        score = rng.choice(["softmax", "sigmoid"])
        return _route(None, T, E, k, dtype, score, rng.random() < 0.6, groups, keep, min(rng.choice([1, 2]), E // groups),
                      rng.random() < 0.5, rng.choice([1.0, 2.5]), pad=rng.choice([0, T // 32]), grad=rng.random() < 0.4)
    if op == "experts":
        E = _spread(rng, 2, 128)
        return _experts(None, _spread(rng, 1, 8192), E, rng.randint(1, min(8, E)), _width(rng, 64, 4096), _width(rng, 64, 4096),
                        dtype, grad=rng.random() < 0.4)
    if op == "combine":
        E = _spread(rng, 2, 128)
        return _combine(None, _spread(rng, 1, 16384), E, rng.randint(1, min(8, E)), _width(rng, 64, 4096), dtype,
                        grad=rng.random() < 0.5)
    T = _spread(rng, 1, 4096)
    return _adapters(None, T, _width(rng, 64, 8192), _width(rng, 64, 8192), rng.choice([4, 8, 16, 16, 24, 32, 64]),
                     _spread(rng, 1, 64), min(T, _spread(rng, 1, 64)), dtype)


def draw(rng):
    """A case of the listed ranges, no dearer than the dearest listed one of its operator."""
    while True:
        c = _drawn(rng)
        del c["name"]
        top = [work(o) for o in listed() if o["op"] == c["op"]]
        if c["dtype"] == "float32":          # the matrix rate is a sixteenth of the 16-bit types'
            top = [work(o) for o in listed() if o["op"] == c["op"] and (o["dtype"] == "float32" or c["op"] != "experts")]
        limit = {q: max(w[q] for w in top) for q in ("bytes", "flops")}
        w = work(c)
        if w["flops"] <= limit["flops"] and w["bytes"] <= limit["bytes"]:
            return c


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def _active(c):
    """Experts that have rows, were the slots spread evenly."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c, z = case, SIZE[case["dtype"]]
    T = c["T"]
    if c["op"] == "route":
        S = T * c["k"]
        b = T * c["E"] * z + (4 * c["E"] if c["bias"] else 0) + 8 * S          # logits, bias; weight and index
        b += 8 * S + 4 * (c["E"] + 1)                                          # order, position, offsets
        f = 2.0 * T * c["E"]
        if c["grad"]:
            b += 4 * S + T * c["E"] * z                                        # dweight; dlogits
            f *= 2
        return {"bytes": int(b), "flops": int(f)}
    if c["op"] == "experts":
        P, K, N = T * c["k"], c["K"], c["N"]
        w = _active(c) * K * N * z
        if not c["grad"]:
            return {"bytes": int(T * K * z + w + P * N * z + 4 * P), "flops": 2 * P * K * N}
        # dY, W in, dX out; X in, dW of every expert out
        return {"bytes": int(P * N * z + w + P * K * z + T * K * z + 4 * P + c["E"] * K * N * z), "flops": 4 * P * K * N}
    if c["op"] == "combine":
        P, N = T * c["k"], c["N"]
        b, f = P * N * z + T * N * z + 8 * P, 2 * P * N
        if c["grad"]:
            b += T * N * z + P * N * z + 4 * P                                 # dout; dY, dweight (Y is already counted)
            f += 3 * P * N
        return {"bytes": int(b), "flops": int(f)}
    K, N, R = c["K"], c["N"], c["R"]
    used = min(c["n"], c["requests"])
    return {"bytes": int((T * K + K * N + T * N + used * R * (K + N)) * z + 4 * T), "flops": 2 * T * K * N + 2 * T * R * (K + N)}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _chosen(g, T, E, k):
    """index [T, k]: k different experts a token, some experts more popular than others."""
    score = _normal(g, T, E) + _normal(g, E, scale=0.7)
    return torch.topk(score, k, dim=1).indices.to(torch.int32).contiguous()


def _places(index, E):
    """offsets (also as a list), order, position of the slots in expert order."""
    flat = index.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=flat.device)
    return offsets.to(torch.int32), offsets.tolist(), order.to(torch.int32), position.reshape(index.shape).to(torch.int32)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = c["T"]
    s = dict(case=c)
    if c["op"] == "route":
        logits = _normal(g, T, c["E"], scale=1.5) + _normal(g, c["E"], scale=0.5)
        if c["pad"]:
            logits[T - c["pad"]:] = -math.inf
        s["logits"] = logits.to(dt)
        s["bias"] = _normal(g, c["E"], scale=0.05) if c["bias"] else None
        if c["grad"]:
            s["dweight"] = _normal(g, T, c["k"])
        return s
    if c["op"] == "experts":
        K, N, E = c["K"], c["N"], c["E"]
        index = _chosen(g, T, E, c["k"])
        s["offsets"], s["bounds"], s["order"], s["position"] = _places(index, E)
        s["X"] = _normal(g, T, K).to(dt)
        s["W"] = torch.empty(E, K, N, device="cuda", dtype=dt)
        for e in range(E):
            s["W"][e] = _normal(g, K, N, scale=K ** -0.5)
        if c["grad"]:
            s["dY"] = _normal(g, T * c["k"], N).to(dt)
        return s
    if c["op"] == "combine":
        index = _chosen(g, T, c["E"], c["k"])
        s["position"] = _places(index, c["E"])[3]
        s["weight"] = torch.softmax(_normal(g, T, c["k"]), 1)
        s["Y"] = _normal(g, T * c["k"], c["N"]).to(dt)
        if c["grad"]:
            s["dout"] = _normal(g, T, c["N"]).to(dt)
        return s
    K, N, R, n, q = c["K"], c["N"], c["R"], c["n"], c["requests"]
    s["X"] = _normal(g, T, K).to(dt)
    s["W"] = _normal(g, K, N, scale=K ** -0.5).to(dt)
    s["A"] = _normal(g, n, K, R, scale=K ** -0.5).to(dt)
    s["B"] = _normal(g, n, R, N, scale=R ** -0.5).to(dt)
    s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    # each request: a stretch of rows, one adapter (or, one in nine, none)
    pick = torch.randint(0, n, (q,), generator=g, device="cuda")
    pick[torch.rand(q, generator=g, device="cuda") < 1.0 / 9] = -1
    if q == T:
        who = torch.arange(T, device="cuda")
    else:
        cuts = torch.randperm(T - 1, generator=g, device="cuda")[:q - 1] + 1
        start = torch.zeros(T, dtype=torch.int64, device="cuda")
        start[cuts] = 1
        who = torch.cumsum(start, 0)
    s["adapter"] = pick[who].to(torch.int32)
    # which rows use which adapter, as the host of a plain loop knows it
    host = s["adapter"].cpu()
    s["rows"] = [(int(a), torch.nonzero(host == a).flatten().cuda()) for a in torch.unique(host).tolist() if a >= 0]
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _select(l, c, bias):
    """Scores (binary64), keys with -inf for what cannot be chosen, index [T, k]."""
    T, E = l.shape
    there = l > -math.inf
    if c["score"] == "softmax":
        top = torch.where(there, l, l.new_full((), -math.inf)).amax(1, keepdim=True)
        top = torch.where(top > -math.inf, top, torch.zeros_like(top))
        e = torch.exp(l - top)
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    both = s + bias.double() if bias is not None else s
    key = both if bias is not None else l
    none = torch.full_like(l, -math.inf)
    key = torch.where(there, key, none)
    if c["groups"] > 1:
        per = E // c["groups"]
        inside = torch.where(there, both, none).view(T, c["groups"], per)
        best = torch.sort(inside, dim=2, descending=True).values[:, :, :c["top"]]
        any_ = best[:, :, 0] > -math.inf
        score = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        score = torch.where(any_, score, torch.full_like(score, -math.inf))
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros(T, c["groups"], dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(per, dim=1), key, none)
    value, index = torch.sort(key, dim=1, descending=True, stable=True)
    value, index = value[:, :c["k"]], index[:, :c["k"]]
    return s, index, value > -math.inf


def _weights(s, index, ok, c):
    w = torch.where(ok, s.gather(1, index), torch.zeros((), dtype=s.dtype, device=s.device))
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return w


def _plain_route(st):
    # scores next to each other decide which expert is taken: 64 bits
    c = st["case"]
    l = st["logits"].double()
    T, E = l.shape
    k = c["k"]
    s, index, ok = _select(l, c, st["bias"])
    w = _weights(s, index, ok, c)
    chosen = torch.where(ok, index, torch.full_like(index, -1))
    flat = chosen.reshape(-1)
    S = flat.numel()
    order = torch.sort(torch.where(flat < 0, torch.full_like(flat, E), flat), stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device).index_add_(0, torch.where(flat < 0, torch.full_like(flat, E), flat), torch.ones_like(flat))
    ends = torch.cumsum(counts[:E], 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    place = torch.empty_like(order)
    place[order] = torch.arange(S, device=l.device)
    position = torch.where(flat < 0, torch.full_like(place, -1), place).view(T, k)
    order = torch.where(torch.arange(S, device=l.device) < offsets[E], order, torch.full_like(order, -1))
    out = [(w * c["scale"]).float(), chosen.int(), offsets.int(), order.int(), position.int()]
    if c["grad"]:
        dw = torch.where(ok, st["dweight"].double(), torch.zeros((), dtype=torch.float64, device=l.device)) * c["scale"]
        sel = torch.where(ok, s.gather(1, index), torch.zeros_like(w))
        if c["normalize"]:
            total = sel.sum(1, keepdim=True)
            ds = torch.where(total > 0, (dw - (w * dw).sum(1, keepdim=True)) / total, torch.zeros_like(dw))
        else:
            ds = dw
        full = torch.zeros_like(l).scatter_add_(1, index, torch.where(ok, ds, torch.zeros_like(ds)))
        if c["score"] == "softmax":
            dl = s * (full - (s * full).sum(1, keepdim=True))
        else:
            dl = full * s * (1.0 - s)
        out.append(dl.to(st["logits"].dtype))
    return out


def _plain_experts(st):
    c, dt = st["case"], st["X"].dtype
    b, order = st["bounds"], st["order"].long()
    P, K, N = order.numel(), c["K"], c["N"]
    if not c["grad"]:
        Y = torch.empty(P, N, device="cuda", dtype=dt)
        for e in range(c["E"]):
            if b[e + 1] > b[e]:
                x = st["X"][order[b[e]:b[e + 1]] // c["k"]].float()
                Y[b[e]:b[e + 1]] = (x @ st["W"][e].float()).to(dt)
        return Y
    dX = torch.empty(P, K, device="cuda", dtype=dt)
    dW = torch.zeros(c["E"], K, N, device="cuda", dtype=dt)
    for e in range(c["E"]):
        if b[e + 1] > b[e]:
            x = st["X"][order[b[e]:b[e + 1]] // c["k"]].float()
            dy = st["dY"][b[e]:b[e + 1]].float()
            dX[b[e]:b[e + 1]] = (dy @ st["W"][e].float().t()).to(dt)
            dW[e] = (x.t() @ dy).to(dt)
    return [dX, dW]


def _plain_combine(st):
    c, dt = st["case"], st["Y"].dtype
    T, k, N = c["T"], c["k"], c["N"]
    rows = st["position"].long()
    y = st["Y"][rows.reshape(-1)].float().view(T, k, N)
    out = [(y * st["weight"][:, :, None]).sum(1).to(dt)]
    if c["grad"]:
        d = st["dout"].float()
        dY = torch.empty_like(st["Y"])
        dY[rows.reshape(-1)] = (d[:, None, :] * st["weight"][:, :, None]).to(dt).view(T * k, N)
        out += [dY, (y * d[:, None, :]).sum(2)]
    return out


def _plain_adapters(st):
    X = st["X"].float()
    y = X @ st["W"].float()
    for a, rows in st["rows"]:
        low = X[rows] @ st["A"][a].float()
        y[rows] += st["scale"][a] * (low @ st["B"][a].float())
    return y.to(st["X"].dtype)


_plain = dict(route=_plain_route, experts=_plain_experts, combine=_plain_combine, adapters=_plain_adapters)


def _own_route(st):
    from dense_fp32_gemm_amd import binding as gb
    c = st["case"]
    w, index = gb.route(st["logits"], c["k"], bias=st["bias"], score=c["score"], groups=c["groups"], keep_groups=c["keep"],
                        group_top=c["top"], normalize=c["normalize"], scale=c["scale"])
    offsets, order, position = gb.expert_map(index, c["E"])
    out = [w, index, offsets, order, position]
    if c["grad"]:
        out.append(gb.route_grad(st["logits"], index, st["dweight"], score=c["score"], normalize=c["normalize"], scale=c["scale"]))
    return out


def _own_experts(st):
    from dense_fp32_gemm_amd import binding as gb
    k = st["case"]["k"]
    if not st["case"]["grad"]:
        return gb.grouped_matmul(st["X"], st["W"], st["offsets"], order=st["order"], per_row=k)
    return [gb.grouped_grad_x(st["dY"], st["W"], st["offsets"]),
            gb.grouped_grad_w(st["X"], st["dY"], st["offsets"], order=st["order"], per_row=k)]


def _own_combine(st):
    from dense_fp32_gemm_amd import binding as gb
    out = [gb.combine(st["Y"], st["position"], st["weight"])]
    if st["case"]["grad"]:
        out += gb.combine_grad(st["dout"], st["Y"], st["position"], st["weight"])
    return out


def _own_adapters(st):
    from dense_fp32_gemm_amd import binding as gb
    return gb.adapter_matmul(st["X"], st["W"], st["A"], st["B"], st["adapter"], st["scale"])


_own = dict(route=_own_route, experts=_own_experts, combine=_own_combine, adapters=_own_adapters)


# --------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms
# --------------------------------------------------------------------------
def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _exact_route(st):
    import numpy as np
    c = st["case"]
    l = st["logits"].double().cpu().numpy()
    T, E = l.shape
    k, per = c["k"], E // c["groups"]
    bias = st["bias"].double().cpu().numpy() if c["bias"] else None
    live = np.isfinite(l).any(axis=1)
    s = np.zeros_like(l)
    with np.errstate(over="ignore"):
        if c["score"] == "softmax":
            p = np.exp(l[live] - l[live].max(axis=1)[:, None])
            s[live] = p / p.sum(axis=1)[:, None]
        else:
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    total = s if bias is None else s + bias
    key = np.where(np.isfinite(l), l if bias is None else total, -np.inf)
    if c["groups"] > 1:
        parts = np.where(np.isfinite(l), total, -np.inf).reshape(T, c["groups"], per)
        best = -np.sort(-parts, axis=2)[:, :, :c["top"]]
        value = np.where(np.isfinite(best), best, 0.0).sum(axis=2)
        value[~np.isfinite(best[:, :, 0])] = -np.inf
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat(rank < c["keep"], per, axis=1), key, -np.inf)
    index = np.argsort(-key, axis=1, kind="stable")[:, :k]
    line = np.arange(T)[:, None]
    ok = np.isfinite(key[line, index])
    w = np.where(ok, s[line, index], 0.0)
    sums = w.sum(axis=1)[:, None]
    unit = w / np.where(sums > 0, sums, 1.0) if c["normalize"] else w
    index = np.where(ok, index, -1)
    flat = index.ravel()
    slots = np.flatnonzero(flat >= 0)
    sorted_slots = slots[np.argsort(flat[slots], kind="stable")]
    order = np.full(T * k, -1)
    order[:slots.size] = sorted_slots
    position = np.full(T * k, -1)
    position[sorted_slots] = np.arange(slots.size)
    offsets = np.searchsorted(flat[sorted_slots], np.arange(E + 1), side="left")
    out = [unit * c["scale"], index.astype(np.int32), offsets.astype(np.int32), order.astype(np.int32), position.reshape(T, k).astype(np.int32)]
    if c["grad"]:
        up = np.where(ok, st["dweight"].double().cpu().numpy(), 0.0) * c["scale"]
        safe = np.maximum(index, 0)
        dl = np.zeros_like(l)
        if c["normalize"]:
            v = unit * (up - (unit * up).sum(axis=1)[:, None])
            if c["score"] == "sigmoid":
                v = v * (1.0 - s[line, safe])
            np.add.at(dl, (np.broadcast_to(line, index.shape)[ok], index[ok]), v[ok])
        elif c["score"] == "sigmoid":
            v = up * w * (1.0 - w)
            np.add.at(dl, (np.broadcast_to(line, index.shape)[ok], index[ok]), v[ok])
        else:
            mean = (w * up).sum(axis=1)[:, None]
            dl = -s * mean
            np.add.at(dl, (np.broadcast_to(line, index.shape)[ok], index[ok]), (w * up)[ok])
        out.append(dl)
    return [torch.from_numpy(np.ascontiguousarray(o)).cuda() for o in out]


def _exact_experts(st):
    c = st["case"]
    owner = torch.searchsorted(st["offsets"].long(), torch.arange(c["T"] * c["k"], device="cuda"), right=True) - 1
    token = torch.div(st["order"].long(), c["k"], rounding_mode="floor")
    if not c["grad"]:
        Y = torch.zeros(owner.numel(), c["N"], dtype=torch.float64, device="cuda")
        for e in torch.unique(owner).tolist():
            mine = torch.nonzero(owner == e).flatten()
            Y[mine] = torch.mm(st["X"].double()[token[mine]], st["W"][e].double())
        return Y
    dX = torch.zeros(owner.numel(), c["K"], dtype=torch.float64, device="cuda")
    dW = torch.zeros(c["E"], c["K"], c["N"], dtype=torch.float64, device="cuda")
    for e in torch.unique(owner).tolist():
        mine = torch.nonzero(owner == e).flatten()
        up = st["dY"].double()[mine]
        dX[mine] = torch.mm(up, st["W"][e].double().t().contiguous())
        dW[e] = torch.mm(st["X"].double()[token[mine]].t().contiguous(), up)
    return [dX, dW]


def _exact_combine(st):
    c = st["case"]
    total = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
    dY = torch.zeros(st["Y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(c["T"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        at = st["position"][:, j].long()
        w = st["weight"][:, j].double().unsqueeze(1)
        y = st["Y"].double()[at]
        total += w * y
        if c["grad"]:
            d = st["dout"].double()
            dY[at] = w * d
            dw[:, j] = torch.linalg.vecdot(y, d)
    return [total, dY, dw] if c["grad"] else [total]


def _exact_adapters(st):
    X = st["X"].double()
    Y = torch.mm(X, st["W"].double())
    which = st["adapter"].long()
    for a in torch.unique(which).tolist():
        if a < 0:
            continue
        mine = torch.nonzero(which == a).flatten()
        wide = torch.mm(st["A"][a].double(), st["B"][a].double()) * st["scale"][a].double()
        Y[mine] += torch.mm(X[mine], wide)
    return Y


_exact = dict(route=_exact_route, experts=_exact_experts, combine=_exact_combine, adapters=_exact_adapters)
