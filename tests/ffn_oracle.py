"""Plain 64-bit implementations (torch, CPU) of the operators of a feed-forward
block, and the error bounds their tests use."""
import math

import torch

from rows_oracle import STEP, TINY, close, product_bound, rows_of  # noqa: F401

INF = math.inf
U = 2.0 ** -24                      # half a step of binary32
# relative error of the gates' binary32 functions: the exponential, reciprocal and products of the sigmoid come to
# less than 5 steps (2^-23) for silu; the others' arguments, up to 90, bring up to 90 half steps more
# (2^x as the hardware gives it is 0 under 2^-126, where the sigmoid's argument v is past 87.3: the sigmoid
# loses up to 2^-126 there, and less the further v goes.  act = g s loses |g| of that, |g| <= 88: 2^-119.  The
# slope s + g s (1 - s) v' loses 1 + |g v'| of it, and v' = kA + 3 kB g^2 <= 3 v / g, |g v'| <= 3 * 88 = 264: 2^-117.
# gelu's own functions underflow no earlier: g p under 13 * 2^-126, p + g e^(-g^2/2) less than 14 * 2^-126.)
LOST_VALUE, LOST_SLOPE = 2.0 ** -119, 2.0 ** -117
GATE_ERROR = {"silu": 2.0 ** -20, "gelu": 2.0 ** -15, "gelu_tanh": 2.0 ** -15}


def summed(X, R):
    """X + R as the type stores it."""
    return X if R is None else (X.double() + R.double()).to(X.dtype)


def rms(S, eps):
    s = S.double()
    n = max(s.shape[1], 1)
    return 1.0 / torch.sqrt((s * s).sum(1, keepdim=True) / n + eps)


def normed(S, weight, eps):
    w = torch.ones(S.shape[1], dtype=torch.float64) if weight is None else weight.double()
    return S.double() * rms(S, eps) * w


def int8_rows(y):
    """(Q, scale) of rows in 64 bits."""
    T, N = y.shape
    Q, scale = torch.zeros(T, N, dtype=torch.int8), torch.zeros(T)
    for t in range(T):
        top = float(y[t].abs().max()) if N and not y[t].isnan().any() else (0.0 if not N else math.nan)
        s = torch.tensor(top / 127.0, dtype=torch.float64).float() if top == top and top != INF else torch.tensor(math.nan)
        s = torch.maximum(s, torch.tensor(2.0 ** -126))
        if not bool(s < INF):
            scale[t] = math.nan
            continue
        scale[t] = s
        Q[t] = torch.round(y[t] / s.double()).clamp(-127, 127).to(torch.int8)
    return Q, scale


def norm_grad(dY, S, weight, eps, dsum):
    """(dX, dweight, bound of dX, sum of the magnitudes of dweight's terms)."""
    d, s = dY.double(), S.double()
    w = torch.ones(s.shape[1], dtype=torch.float64) if weight is None else weight.double()
    r = rms(S, eps)
    n = max(s.shape[1], 1)
    m = (w * d * s).sum(1, keepdim=True) / n
    size = (w * d * s).abs().sum(1, keepdim=True) / n
    extra = torch.zeros_like(s) if dsum is None else dsum.double()
    dX = r * (w * d - s * r * r * m) + extra
    # each of r, w d, k = r^2 m (whose terms w d are rounded), the difference and the product: half a step
    err = 8 * U * r * ((w * d).abs() + s.abs() * r * r * size) + U * (dX.abs() + extra.abs())
    return dX, (d * s * r).sum(0), err + STEP[dY.dtype] * (dX.abs() + err) + TINY[dY.dtype], (d * s * r).abs().sum(0)


def gate(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    if kind == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    return g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3))


def gate_parts(g, kind):
    """p and p' g of act(g) = g p(g), whose derivative is their sum."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return s, g * s * torch.sigmoid(-g)
    if kind == "gelu":
        return 0.5 * torch.erfc(-g / math.sqrt(2.0)), g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    v = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    return torch.sigmoid(v), g * torch.sigmoid(v) * torch.sigmoid(-v) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g * g)


def int8_product(Q, scale, W, w_scale, bias, dtype):
    """(Y, bound): the sums exact, a rounding to binary32, the scales' product, theirs, and the bias."""
    Y = (Q.double() @ W.double().t()) * scale.double()[:, None] * w_scale.double()
    b = torch.zeros(W.shape[0], dtype=torch.float64) if bias is None else bias.double()
    err = 4 * U * Y.abs() + U * (Y + b).abs() + 2.0 ** -126
    want = Y + b
    return want, err + STEP[dtype] * (want.abs() + err) + TINY[dtype]


def gated(rows, W, kind, dtype):
    """(H, bound, pre, bound) of rows [P, K] in 64 bits and W [K, 2 N]."""
    N, K = W.shape[1] // 2, W.shape[0]
    pre = rows @ W.double()
    mag = rows.abs() @ W.double().abs()
    g, u = pre[:, :N], pre[:, N:]
    err = 2.0 * K * 2.0 ** -23 * mag
    eg, eu = err[:, :N], err[:, N:]
    a = gate(g, kind)
    H = a * u
    # the gates' slope is under 1.2 everywhere
    e = 1.2 * eg * (u.abs() + eu) + a.abs() * eu + (GATE_ERROR[kind] + 2 * U) * (a.abs() + 1.2 * eg) * (u.abs() + eu) + LOST_VALUE * (1 + u.abs())
    return H, e + STEP[dtype] * (H.abs() + e) + TINY[dtype], pre, product_bound(pre, mag, K, dtype)


def gate_grad(dH, pre, kind):
    """(dpre, bound)."""
    N = dH.shape[1]
    d, g, u = dH.double(), pre[:, :N].double(), pre[:, N:].double()
    p, q = gate_parts(g, kind)
    want = torch.cat([d * u * (p + q), d * g * p], 1)
    size = torch.cat([(d * u).abs() * (p.abs() + q.abs()), (d * g * p).abs()], 1)
    err = (GATE_ERROR[kind] + 4 * U) * size + 2.0 ** -126
    err = err + torch.cat([LOST_SLOPE * (d * u).abs(), LOST_VALUE * d.abs()], 1)
    return want, err + STEP[dH.dtype] * (want.abs() + err) + TINY[dH.dtype]
