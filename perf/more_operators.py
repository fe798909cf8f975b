"""Cases of the operators of a feed-forward block.

The root-mean-square norm with the residual's addition and its gradient; 8-bit
projections, whose input comes from that norm, from a gated pair of
projections or as it is, with a scale for each token and channel; and the
gated pair of projections, dense or by expert, with its gradients.  `listed`
and `draw` say what is run, `prepare` makes the tensors a program holds before
the call, `run` makes one pass: in plain torch operations, or (`own`) through
dense_fp32_gemm_amd.binding.  `exact` computes the same outputs from the
definitions in binary64.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
EPS = 1e-6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _norm(name, T, N, dtype, residual, grad=False):
    return dict(name=name, op="norm", T=T, N=N, dtype=dtype, residual=residual, grad=grad)


def _project(name, T, K, N, dtype, source, gate="silu", residual=False, bias=False):
    return dict(name=name, op="project", T=T, K=K, N=N, dtype=dtype, source=source, gate=gate, residual=residual, bias=bias)


def _gated(name, T, E, k, K, N, dtype, gate="silu", save=False, grad=False):
    return dict(name=name, op="gated", T=T, E=E, k=k, K=K, N=N, dtype=dtype, gate=gate, save=save, grad=grad)


def listed():
    return [
        # one decoding step of a small batch: latency
        _norm("norm_step", 16, 4096, "bfloat16", True),
        # a long prompt batch
        _norm("norm_prompt", 8192, 4096, "float16", True),
        # a training batch with an odd number of rows: gradients of the row and of the weight, the residual's added
        _norm("norm_train", 16383, 2048, "bfloat16", True, grad=True),
        # one decoding step through an 8-bit projection: norm, 8-bit rows, product; the weights are what is read
        _project("project_step", 16, 4096, 4096, "bfloat16", "norm", residual=True),
        # a single token through an 8-bit down-projection behind the gate
        _project("down_step", 1, 8192, 2048, "bfloat16", "gate"),
        # a long prompt batch through an 8-bit projection
        _project("project_prompt", 8192, 4096, 4096, "bfloat16", "norm", residual=True),
        # a prompt batch through the down-projection behind the gate
        _project("down_prompt", 4096, 8192, 4096, "float16", "gate"),
        # sizes that fit no tile, rows as they are, results in binary32
        _project("project_odd", 1025, 1000, 1023, "float32", "rows", bias=True),
        # one decoding step: 32 slots over 32 experts, the weights of the chosen experts are what is read
        _gated("gated_step", 8, 32, 4, 2048, 1024, "bfloat16"),
        # a long prompt batch through a dense block, the pre-activations kept for the gradient
        _gated("gated_prompt", 8192, 1, 1, 2048, 4096, "bfloat16", "gelu_tanh", save=True),
        # training of experts: gradients of the rows and of the weights
        _gated("gated_train", 4096, 16, 4, 2048, 1024, "bfloat16", grad=True),
        # training of a dense block in binary32 with sizes that fit no tile
        _gated("gated_train_odd", 1025, 1, 1, 1000, 1023, "float32", "gelu", grad=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A row length: mostly a multiple of 64, else any number."""
    w = _spread(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def _drawn(rng):
    op = rng.choice(["norm", "project", "project", "gated", "gated"])
    dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
    gate = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    if op == "norm":
        return _norm(None, _spread(rng, 1, 16384), _width(rng, 64, 8192), dtype, rng.random() < 0.7, grad=rng.random() < 0.5)
    if op == "project":
        source = rng.choice(["norm", "gate", "rows"])
        return _project(None, _spread(rng, 1, 8192), _width(rng, 64, 8192), _width(rng, 64, 8192), dtype, source, gate,
                        source == "norm" and rng.random() < 0.7, rng.random() < 0.3)
    E = 1 if rng.random() < 0.5 else _spread(rng, 2, 64)
    grad = rng.random() < 0.4
    return _gated(None, _spread(rng, 1, 8192), E, rng.randint(1, min(8, E)), _width(rng, 64, 4096), _width(rng, 64, 4096), dtype,
                  gate, not grad and rng.random() < 0.4, grad)


def draw(rng):
    """A case of the listed ranges, no dearer than the dearest listed one of its operator."""
    while True:
        c = _drawn(rng)
        del c["name"]
        top = [work(o) for o in listed() if o["op"] == c["op"]]
        if c["op"] == "gated" and c["dtype"] == "float32":          # the matrix rate is a sixteenth of the 16-bit types'
            top = [dict(w, flops=w["flops"] / 8) for w in top]
        limit = {q: max(w[q] for w in top) for q in ("bytes", "flops")}
        w = work(c)
        if w["flops"] <= limit["flops"] and w["bytes"] <= limit["bytes"]:
            return c


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c, z = case, SIZE[case["dtype"]]
    T, N = c["T"], c["N"]
    if c["op"] == "norm":
        if c["grad"]:                                # dY, S (and dS) in, dX out; weight and its gradient
            return {"bytes": T * N * z * (4 if c["residual"] else 3) + 8 * N, "flops": 10 * T * N}
        return {"bytes": T * N * z * (4 if c["residual"] else 2) + 4 * N, "flops": 5 * T * N}
    K = c["K"]
    if c["op"] == "project":
        rows = {"norm": 3 if c["residual"] else 1, "gate": 2, "rows": 1}[c["source"]]
        b = rows * T * K * z + N * K + T * N * z + 4 * N + (4 * K if c["source"] == "norm" else 0) + (4 * N if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * K * N}
    P, E = T * c["k"], c["E"]
    active = E * (1.0 - (1.0 - c["k"] / E) ** T)     # experts that have rows, were the slots spread evenly
    listing = 4 * P if E > 1 else 0
    if c["grad"]:
        # dH, pre, X, W in; dX, dW of every expert out
        return {"bytes": int(3 * P * N * z + T * K * z + active * 2 * K * N * z + P * K * z + E * 2 * K * N * z + listing),
                "flops": 8 * P * K * N}
    return {"bytes": int(T * K * z + active * 2 * K * N * z + P * N * z * (3 if c["save"] else 1) + listing), "flops": 4 * P * K * N}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _hidden(g, T, N):
    """Rows as a model's residual stream has them: rows of unlike size, a few channels that stand out."""
    loud = 1.0 + 9.0 * (torch.rand(N, generator=g, device="cuda") < 0.01)
    return _normal(g, T, N) * loud * torch.exp(_normal(g, T, 1, scale=0.5))


def _places(index, E):
    """offsets (also as a list) and order of the slots in expert order."""
    flat = index.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return offsets.to(torch.int32), offsets.tolist(), order.to(torch.int32)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, N = c["T"], c["N"]
    s = dict(case=c)
    if c["op"] == "norm":
        s["X"] = _hidden(g, T, N).to(dt)             # of a gradient: the sum that the forward pass stored
        s["R"] = _normal(g, T, N).to(dt) if c["residual"] else None
        s["weight"] = 1.0 + _normal(g, N, scale=0.1)
        if c["grad"]:
            s["dY"] = _normal(g, T, N).to(dt)
        return s
    K = c["K"]
    if c["op"] == "project":
        if c["source"] == "norm":
            s["X"] = _hidden(g, T, K).to(dt)
            s["R"] = _normal(g, T, K).to(dt) if c["residual"] else None
            s["weight"] = 1.0 + _normal(g, K, scale=0.1)
        elif c["source"] == "gate":
            s["X"] = _normal(g, T, 2 * K).to(dt)
        else:
            s["X"] = _hidden(g, T, K).to(dt)
        W = _normal(g, N, K, scale=K ** -0.5)        # a channel a row, as it is kept in 8 bits
        s["W_scale"] = W.abs().amax(1) / 127.0
        s["W"] = torch.round(W / s["W_scale"][:, None]).clamp(-127, 127).to(torch.int8)
        s["bias"] = _normal(g, N, scale=0.1) if c["bias"] else None
        return s
    E, k = c["E"], c["k"]
    s["offsets"], s["bounds"], s["order"] = None, [0, T], None
    if E > 1:
        # k different experts a token, some more popular than others
        index = torch.topk(_normal(g, T, E) + _normal(g, E, scale=0.7), k, dim=1).indices
        s["offsets"], s["bounds"], s["order"] = _places(index, E)
    s["X"] = _normal(g, T, K).to(dt)
    s["W"] = torch.empty(E, K, 2 * N, device="cuda", dtype=dt)     # an expert's gate, then what it gates
    for e in range(E):
        s["W"][e] = _normal(g, K, 2 * N, scale=K ** -0.5)
    if c["grad"]:
        s["pre"] = _normal(g, T * k, 2 * N).to(dt)   # what the forward pass kept
        s["dH"] = _normal(g, T * k, N).to(dt)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _summed(X, R):
    """X + R as it is stored, in X's type."""
    return X if R is None else (X.float() + R.float()).to(X.dtype)


def _plain_norm(st):
    c, dt = st["case"], st["X"].dtype
    if not c["grad"]:
        S = _summed(st["X"], st["R"])
        z = S.float()
        Y = (z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * st["weight"]).to(dt)
        return [Y, S] if c["residual"] else [Y]
    s, d = st["X"].float(), st["dY"].float()
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
    wd = d * st["weight"]
    dX = r * (wd - s * (r * r * (wd * s).mean(1, keepdim=True)))
    if c["residual"]:
        dX = dX + st["R"].float()
    return [dX.to(dt), (d * s * r).sum(0)]


def _activation(g, gate):
    if gate == "silu":
        return g / (1.0 + torch.exp(-g))
    if gate == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 2.0 ** -0.5))
    return 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g)))


def _slope(g, gate):
    if gate == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if gate == "gelu":
        return 0.5 * (1.0 + torch.erf(g * 2.0 ** -0.5)) + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    a = (2.0 / math.pi) ** 0.5
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_project(st):
    # 8-bit values next to a rounding border, and whole sums over 2^24: 64 bits
    c, dt = st["case"], st["X"].dtype
    K = c["K"]
    out = []
    if c["source"] == "norm":
        S = _summed(st["X"], st["R"])
        z = S.double()
        y = z / torch.sqrt((z * z).mean(1, keepdim=True) + EPS) * st["weight"].double()
        if c["residual"]:
            out.append(S)
    elif c["source"] == "gate":
        z = st["X"].double()
        y = _activation(z[:, :K], c["gate"]) * z[:, K:]
    else:
        y = st["X"].double()
    scale = (y.abs().amax(1, keepdim=True) / 127.0).float().clamp_min(2.0 ** -126)
    q = torch.round(y / scale.double()).clamp(-127, 127)
    Y = (q @ st["W"].double().t()) * scale.double() * st["W_scale"].double()
    if c["bias"]:
        Y = Y + st["bias"].double()
    return [Y.to(dt)] + out


def _rows(st, e):
    """Places of expert e, and their rows of X in binary32."""
    lo, hi = st["bounds"][e], st["bounds"][e + 1]
    x = st["X"][lo:hi] if st["order"] is None else st["X"][st["order"][lo:hi].long() // st["case"]["k"]]
    return lo, hi, x.float()


def _plain_gated(st):
    c, dt = st["case"], st["X"].dtype
    P, K, N, E = c["T"] * c["k"], c["K"], c["N"], c["E"]
    if not c["grad"]:
        H = torch.empty(P, N, device="cuda", dtype=dt)
        pre = torch.empty(P, 2 * N, device="cuda", dtype=dt) if c["save"] else None
        for e in range(E):
            lo, hi, x = _rows(st, e)
            if hi > lo:
                gu = x @ st["W"][e].float()
                H[lo:hi] = (_activation(gu[:, :N], c["gate"]) * gu[:, N:]).to(dt)
                if c["save"]:
                    pre[lo:hi] = gu.to(dt)
        return [H, pre] if c["save"] else [H]
    dX = torch.empty(P, K, device="cuda", dtype=dt)
    dW = torch.zeros(E, K, 2 * N, device="cuda", dtype=dt)
    for e in range(E):
        lo, hi, x = _rows(st, e)
        if hi > lo:
            g, u, d = st["pre"][lo:hi, :N].float(), st["pre"][lo:hi, N:].float(), st["dH"][lo:hi].float()
            dgu = torch.cat([d * u * _slope(g, c["gate"]), d * _activation(g, c["gate"])], 1)
            dX[lo:hi] = (dgu @ st["W"][e].float().t()).to(dt)
            dW[e] = (x.t() @ dgu).to(dt)
    return [dX, dW]


_plain = dict(norm=_plain_norm, project=_plain_project, gated=_plain_gated)


def _own_norm(st):
    from dense_fp32_gemm_amd import binding as gb
    c = st["case"]
    if c["grad"]:
        return list(gb.rms_norm_grad(st["dY"], st["X"], st["weight"], eps=EPS, dsum=st["R"]))
    out = gb.rms_norm(st["X"], st["weight"], eps=EPS, residual=st["R"])
    return list(out) if c["residual"] else [out]


def _own_project(st):
    from dense_fp32_gemm_amd import binding as gb
    c = st["case"]
    out = []
    if c["source"] == "norm":
        Q, scale, *out = gb.rms_norm_int8(st["X"], st["weight"], eps=EPS, residual=st["R"])
    else:
        Q, scale = gb.quantize(st["X"], gate=c["gate"] if c["source"] == "gate" else None)
    return [gb.int8_matmul(Q, scale, st["W"], st["W_scale"], bias=st["bias"], dtype=st["X"].dtype), *out]


def _own_gated(st):
    from dense_fp32_gemm_amd import binding as gb
    c = st["case"]
    if not c["grad"]:
        out = gb.gated_matmul(st["X"], st["W"], st["offsets"], order=st["order"], per_row=c["k"], gate=c["gate"], save=c["save"])
        return list(out) if c["save"] else [out]
    dpre = gb.gate_grad(st["dH"], st["pre"], gate=c["gate"])
    return [gb.grouped_grad_x(dpre, st["W"], st["offsets"]),
            gb.grouped_grad_w(st["X"], dpre, st["offsets"], order=st["order"], per_row=c["k"])]


_own = dict(norm=_own_norm, project=_own_project, gated=_own_gated)


# --------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms
# --------------------------------------------------------------------------
def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _stored(st):
    """The sum in 64 bits, as the type that stores it rounds it."""
    if st["R"] is None:
        return st["X"].double()
    return torch.add(st["X"].double(), st["R"].double()).to(st["X"].dtype).double()


def _exact_norm(st):
    c = st["case"]
    w = st["weight"].double()
    if not c["grad"]:
        s = _stored(st)
        Y = torch.empty_like(s)
        for lo in range(0, c["T"], 4096):
            rows = s[lo:lo + 4096]
            power = torch.linalg.vecdot(rows, rows) / c["N"] + EPS
            Y[lo:lo + 4096] = rows * w / power.sqrt().unsqueeze(1)
        return [Y, s] if c["residual"] else [Y]
    dX, dw = [], torch.zeros_like(w)
    for lo in range(0, c["T"], 4096):
        s, d = st["X"][lo:lo + 4096].double(), st["dY"][lo:lo + 4096].double()
        size = (torch.linalg.vecdot(s, s) / c["N"] + EPS).sqrt().unsqueeze(1)
        n = s / size                                 # the normalised row: dX is what of w dY is not along it, nearly
        along = torch.linalg.vecdot(d * w, n).unsqueeze(1) / c["N"]
        g = (d * w - n * along) / size
        dX.append(g + st["R"][lo:lo + 4096].double() if c["residual"] else g)
        dw += torch.linalg.vecdot(d.t(), n.t())
    return [torch.cat(dX), dw]


def _exact_gate(g, gate):
    """The activation and its derivative."""
    if gate == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if gate == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    v = math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)         # (1 + tanh(v / 2)) / 2 = 1 / (1 + exp(-v))
    s = torch.sigmoid(v)
    return g * s, s + g * s * (1 - s) * math.sqrt(8.0 / math.pi) * (1 + 0.134145 * g ** 2)


def _exact_project(st):
    c = st["case"]
    Wf = st["W"].double() * st["W_scale"].double().unsqueeze(1)
    out, sums = [], _stored(st) if c["source"] == "norm" else None
    for lo in range(0, c["T"], 2048):
        if c["source"] == "norm":
            s = sums[lo:lo + 2048]
            y = s * st["weight"].double() * (torch.linalg.vecdot(s, s) / c["K"] + EPS).rsqrt().unsqueeze(1)
        elif c["source"] == "gate":
            g, u = st["X"][lo:lo + 2048].double().split(c["K"], dim=1)
            y = _exact_gate(g, c["gate"])[0] * u
        else:
            y = st["X"][lo:lo + 2048].double()
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1, keepdim=True).div(127.0).to(torch.float32).double().clamp_min(2.0 ** -126)
        out.append(torch.mm((y / step).round().clamp(-127, 127) * step, Wf.t().contiguous()))
    Y = torch.cat(out)
    if c["bias"]:
        Y += st["bias"].double()
    return [Y, sums] if c["source"] == "norm" and c["residual"] else [Y]


def _exact_gated(st):
    c = st["case"]
    P, K, N = c["T"] * c["k"], c["K"], c["N"]
    place = torch.arange(P, device="cuda")
    if st["order"] is None:
        owner, token = torch.zeros_like(place), place
    else:
        owner = torch.searchsorted(st["offsets"].long(), place, right=True) - 1
        token = torch.div(st["order"].long(), c["k"], rounding_mode="floor")
    a = torch.zeros(P, K if c["grad"] else N, dtype=torch.float64, device="cuda")
    b = torch.zeros((c["E"], K, 2 * N) if c["grad"] else (P, 2 * N), dtype=torch.float64, device="cuda")
    for e in torch.unique(owner).tolist():
        mine = torch.nonzero(owner == e).flatten()
        x = st["X"].double()[token[mine]]
        up, gate = st["W"][e][:, N:].double(), st["W"][e][:, :N].double()
        if not c["grad"]:
            g, u = torch.mm(x, gate), torch.mm(x, up)
            a[mine] = _exact_gate(g, c["gate"])[0] * u
            b[mine, :N], b[mine, N:] = g, u
            continue
        f, slope = _exact_gate(st["pre"][mine, :N].double(), c["gate"])
        dg = st["dH"][mine].double() * st["pre"][mine, N:].double() * slope
        du = st["dH"][mine].double() * f
        a[mine] = torch.mm(dg, gate.t().contiguous()) + torch.mm(du, up.t().contiguous())
        b[e, :, :N], b[e, :, N:] = torch.mm(x.t().contiguous(), dg), torch.mm(x.t().contiguous(), du)
    return [a, b] if c["grad"] or c["save"] else [a]


_exact = dict(norm=_exact_norm, project=_exact_project, gated=_exact_gated)
