"""The row-chosen products on the GPU against plain 64-bit implementations
(rows_oracle.py).  Whole numbers are equal; sums are within the bound of binary32 summation plus
one rounding to the output's type (rows_oracle.product_bound)."""
import math
import sys
import zlib

import pytest

from dense_fp32_gemm_amd import binding as gb
import rows_oracle as oracle

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def say(*msg):
    print("[rows]", *msg, file=sys.__stderr__, flush=True)


def seeded(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def strided(t, pad, dev, fill=NAN):
    """A copy on the GPU whose rows are `pad` elements further apart, filled around."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype)
    wide[..., :t.shape[-1]] = t
    return wide.to(dev)[..., :t.shape[-1]]


# --- routing ---------------------------------------------------------------------
ROUTES = [
    # T, E, k, options
    (1, 1, 1, dict()), (1, 2, 2, dict(normalize=True)), (7, 8, 2, dict(score="sigmoid")), (33, 64, 4, dict(normalize=True, scale=2.5)),
    (5, 65, 8, dict()), (9, 128, 6, dict(score="sigmoid", normalize=True, bias=True)), (6, 100, 64, dict(normalize=True)),
    (11, 256, 8, dict(score="sigmoid", normalize=True, bias=True, groups=8, keep_groups=4, group_top=2, scale=2.5)),
    (10, 160, 6, dict(groups=8, keep_groups=3, group_top=1)), (4, 512, 8, dict(bias=True)), (3, 1024, 10, dict(normalize=True)),
    (3, 1000, 5, dict(score="sigmoid", bias=True, groups=40, keep_groups=7, group_top=2)),
    (12, 64, 3, dict(groups=64, keep_groups=5, group_top=2, score="sigmoid", normalize=True)),
    (8, 12, 12, dict(groups=4, keep_groups=2, group_top=2, bias=True, normalize=True)),
    # many tokens: four to a wave
    (1025, 40, 4, dict(normalize=True)), (1030, 100, 16, dict(score="sigmoid", bias=True)), (4099, 256, 8, dict()),
    (4097, 200, 8, dict(score="sigmoid", normalize=True, bias=True, groups=10, keep_groups=4, group_top=2)),
    (1026, 120, 3, dict(groups=8, keep_groups=2, group_top=1, normalize=True)),
]


def masked_logits(g, T, E, dtype):
    """Rows of each kind: ordinary, ties, masked in part, wholly, at the type's lowest value, +inf, NaN."""
    l = normal(g, T, E, scale=1.5)
    for t in range(T):
        kind = t % 7
        if kind == 1:
            l[t] = torch.round(l[t])                            # ties
        elif kind == 2:
            l[t, torch.rand(E, generator=g) < 0.6] = -INF
        elif kind == 3:
            l[t] = -INF
        elif kind == 4:
            l[t, torch.rand(E, generator=g) < 0.7] = torch.finfo(dtype).min
        elif kind == 5:
            l[t, E // 2] = INF
            l[t, 0] = -INF if E > 1 else 0.0
        elif kind == 6:
            l[t, E // 3] = NAN
    return l.to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(dev, dtype, case):
    T, E, k, opt = ROUTES[case]
    opt = dict(opt)
    g = seeded("route", case)
    l = masked_logits(g, T, E, dtype)
    bias = normal(g, E, scale=0.1) if opt.pop("bias", False) else None
    if bias is not None and E > 4:
        bias[E // 4] = -INF
    say("route", T, E, k, opt, dtype)
    want_w, want_i, _ = oracle.route(l, k, bias=bias, **opt)
    w, i = gb.route(strided(l, 3, dev), k, bias=None if bias is None else bias.to(dev), **opt)
    assert torch.equal(i.cpu(), want_i)
    # binary64 throughout (a few 2^-52 over at most 1024 terms), one rounding to binary32
    oracle.close(w, want_w, want_w.abs() * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150, "weight")


GRADS = [(1, 1, 1), (9, 8, 2), (14, 65, 8), (7, 256, 8), (7, 1000, 64), (1031, 50, 3), (1025, 128, 16), (4098, 200, 8)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T,E,k", GRADS)
def test_route_grad(dev, dtype, score, normalize, T, E, k):
    g = seeded("grad", T, E, k)
    l = normal(g, T, E, scale=1.5)
    if T > 4 and E > 2:
        l[1, torch.rand(E, generator=g) < 0.5] = -INF
        l[2] = -INF
        l[3, ::2] = torch.finfo(dtype).min
    l = l.to(dtype)
    dw = normal(g, T, k)
    say("route_grad", T, E, k, score, normalize, dtype)
    _, index, _ = oracle.route(l, k, score=score, normalize=normalize, scale=1.5)
    want = oracle.route_grad(l, index, dw, score, normalize, 1.5)
    full = torch.full((T, E + 5), 7.0, dtype=dtype, device=dev)
    gb.route_grad(strided(l, 2, dev), index.to(dev), dw.to(dev), score=score, normalize=normalize, scale=1.5, out=full[:, :E])
    assert (full[:, E:] == 7.0).all()
    # both sides in binary64; their terms cancel to within 2^-52 of the row's largest dweight
    room = 2.0 ** -44 * 1.5 * dw.double().abs().sum(1, keepdim=True)
    oracle.close(full[:, :E], want, want.abs() * (oracle.STEP[dtype] + 2.0 ** -23) + room + oracle.TINY[dtype], "dlogits")


def test_route_grad_adds_what_an_index_named_twice_gets(dev):
    l = normal(seeded("twice"), 2, 6).to(dev)
    dw = torch.tensor([[1.0, 2.0], [3.0, 4.0]], device=dev)
    once = gb.route_grad(l, torch.tensor([[3, -1], [9, 2]], dtype=torch.int32, device=dev), dw, score="sigmoid")
    s = torch.sigmoid(l.double())
    want = torch.zeros(2, 6, dtype=torch.float64, device=dev)
    want[0, 3] = (s * (1 - s))[0, 3]
    want[1, 2] = 4 * (s * (1 - s))[1, 2]
    oracle.close(once, want.cpu(), want.cpu().abs() * 2.0 ** -23, "skipped")
    both = gb.route_grad(l, torch.tensor([[3, 3], [1, 1]], dtype=torch.int32, device=dev), dw, score="sigmoid")
    want.zero_()
    want[0, 3] = 3 * (s * (1 - s))[0, 3]
    want[1, 1] = 7 * (s * (1 - s))[1, 1]
    oracle.close(both, want.cpu(), want.cpu().abs() * 2.0 ** -23, "twice")


@pytest.mark.parametrize("S,E", [(0, 3), (1, 1), (5, 4), (64, 64), (2047, 7), (2048, 1024), (2049, 3), (6000, 130), (20001, 1000), (32768, 9),
                                 (32769, 64), (150001, 256), (1 << 17, 130), ((1 << 18) - 2048, 5), (1 << 18, 130), ((1 << 19) + 33, 7), (4000001, 1024)])
def test_expert_map(dev, S, E):
    g = seeded("map", S, E)
    index = torch.randint(-1, E + 1, (S,), generator=g, dtype=torch.int32)      # -1 and E: left out
    index[S // 2:] = torch.where(torch.rand(S - S // 2, generator=g) < 0.5, torch.zeros((), dtype=torch.int32), index[S // 2:])
    say("expert_map", S, E)
    for got, want in zip(gb.expert_map(index.to(dev), E), oracle.expert_map(index, E)):
        assert torch.equal(got.cpu(), want)


# --- products per group ------------------------------------------------------------
def places(g, T, k, E, drop=0.0):
    """offsets, order, position of a random choice, some slots left out, some experts without any."""
    score = torch.rand(T, E, generator=g)
    score[:, E // 2] = -1.0
    index = torch.topk(score, k, dim=1).indices.int()
    index[torch.rand(T, k, generator=g) < drop] = -1
    return oracle.expert_map(index, E)


SHAPES = [
    # T, E, k, K, N
    (1, 1, 1, 1, 1), (1, 4, 2, 8, 8), (5, 3, 1, 17, 33), (3, 8, 4, 64, 128), (40, 4, 2, 65, 63), (33, 70, 2, 96, 136),
    (200, 3, 2, 129, 200), (300, 2, 2, 72, 256), (260, 5, 3, 256, 24), (9, 2, 1, 0, 5), (513, 2, 1, 128, 130), (700, 130, 2, 64, 64),
]


def grouped_want(X, W, offsets, order, k):
    rows = oracle.rows_of(X, order, k)
    want = torch.zeros(len(order), W.shape[2], dtype=torch.float64)
    size = torch.zeros_like(want)
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[lo:hi] = rows[lo:hi] @ W[e].double()
        size[lo:hi] = rows[lo:hi].abs() @ W[e].double().abs()
    return want, size


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T,E,k,K,N", SHAPES)
def test_grouped_and_its_gradients(dev, dtype, pad, T, E, k, K, N):
    g = seeded("grouped", T, E, k, K, N)
    offsets, order, position = places(g, T, k, E, drop=0.1)
    P, used = len(order), int(offsets[-1])
    X, W = normal(g, T, K, dtype=dtype), normal(g, E, K, N, dtype=dtype, scale=max(K, 1) ** -0.5)
    dY = normal(g, P, N, dtype=dtype)
    say("grouped", T, E, k, K, N, pad, dtype)
    dX, dW_, dYd = strided(X, pad, dev), strided(W, pad, dev), strided(dY, pad, dev)
    off, ord_ = offsets.to(dev), order.to(dev)

    full = torch.full((P, N + pad), 7.0, dtype=dtype, device=dev)
    gb.grouped_matmul(dX, dW_, off, order=ord_, per_row=k, out=full[:, :N])
    want, size = grouped_want(X, W, offsets, order, k)
    oracle.close(full[:used, :N], want[:used], oracle.product_bound(want, size, K + 1, dtype)[:used], "Y")
    assert (full[used:] == 7.0).all() and (full[:, N:] == 7.0).all()

    full = torch.full((P, K + pad), 7.0, dtype=dtype, device=dev)
    gb.grouped_grad_x(dYd, dW_, off, out=full[:, :K])
    want, size = torch.zeros(P, K, dtype=torch.float64), torch.zeros(P, K, dtype=torch.float64)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[lo:hi] = dY[lo:hi].double() @ W[e].double().t()
        size[lo:hi] = dY[lo:hi].double().abs() @ W[e].double().abs().t()
    oracle.close(full[:used, :K], want[:used], oracle.product_bound(want, size, N + 1, dtype)[:used], "dX")
    assert (full[used:] == 7.0).all() and (full[:, K:] == 7.0).all()

    full = torch.full((E, K, N + pad), 7.0, dtype=dtype, device=dev)
    gb.grouped_grad_w(dX, dYd, off, order=ord_, per_row=k, out=full[:, :, :N])
    rows = oracle.rows_of(X, order, k)
    want, size = torch.zeros(E, K, N, dtype=torch.float64), torch.zeros(E, K, N, dtype=torch.float64)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want[e] = rows[lo:hi].t() @ dY[lo:hi].double()
        size[e] = rows[lo:hi].t().abs() @ dY[lo:hi].double().abs()
    oracle.close(full[:, :, :N], want, oracle.product_bound(want, size, P + 1, dtype), "dW")
    assert (full[:, :, N:] == 7.0).all()


def close_on_gpu(got, want, size, terms, what):
    """oracle.product_bound, evaluated where the (large) tensors are."""
    bound = oracle.product_bound(want, size, terms, got.dtype)
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,E,k,K,N", [(1900, 3, 2, 40, 2500), (2000, 2, 2, 24, 4400), (2300, 4, 2, 72, 4400), (520, 2, 1, 700, 600)])
def test_grouped_large_tiles_whole_and_cut(dev, dtype, T, E, k, K, N):
    """Enough tiles for the large kinds: whole rounds, and a last round cut into two and four."""
    g = seeded("large", T, E, k, K, N)
    offsets, order, position = places(g, T, k, E)
    X, W = normal(g, T, K, dtype=dtype).to(dev), normal(g, E, K, N, dtype=dtype).to(dev)
    dY = normal(g, T * k, N, dtype=dtype).to(dev)
    off, ord_ = offsets.to(dev), order.to(dev)
    say("large tiles", T, E, k, K, N, dtype)
    Y = gb.grouped_matmul(X, W, off, order=ord_, per_row=k)
    dX = gb.grouped_grad_x(dY, W, off)
    dW = gb.grouped_grad_w(X, dY, off, order=ord_, per_row=k)
    rows = X.double()[torch.div(ord_.long(), k, rounding_mode="floor")]
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        x, w, d = rows[lo:hi], W[e].double(), dY[lo:hi].double()
        close_on_gpu(Y[lo:hi], torch.mm(x, w), torch.mm(x.abs(), w.abs()), K + 1, "Y")
        close_on_gpu(dX[lo:hi], torch.mm(d, w.t().contiguous()), torch.mm(d.abs(), w.abs().t().contiguous()), N + 1, "dX")
        close_on_gpu(dW[e], torch.mm(x.t().contiguous(), d), torch.mm(x.abs().t().contiguous(), d.abs()), hi - lo + 1, "dW")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("K,N", [(64, 136), (77, 61)])
def test_grouped_without_order_and_rows_out_of_range(dev, dtype, K, N):
    g = seeded("plain groups", K, N)
    sizes = [0, 150, 1, 0, 17, 129, 0]
    offsets = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)
    P = int(offsets[-1])
    X, W = normal(g, P, K, dtype=dtype), normal(g, len(sizes), K, N, dtype=dtype)
    identity = torch.arange(P, dtype=torch.int32)
    want, size = grouped_want(X, W, offsets, identity, 1)
    say("grouped without order", dtype, K, N)
    got = gb.grouped_matmul(X.to(dev), W.to(dev), offsets.to(dev))
    oracle.close(got, want, oracle.product_bound(want, size, K + 1, dtype), "Y")
    wild = identity.clone()
    wild[3], wild[60], wild[-1] = -5, P, 2 ** 31 - 1            # zero rows
    want, size = grouped_want(X, W, offsets, wild, 1)
    got = gb.grouped_matmul(X.to(dev), W.to(dev), offsets.to(dev), order=wild.to(dev))
    oracle.close(got, want, oracle.product_bound(want, size, K + 1, dtype), "zero rows")
    # offsets outside 0..P are clamped: nothing outside the operands is touched
    far = torch.tensor([-7, 0, 150, 151, 151, 168, 297 + 1000, 9 * P], dtype=torch.int32)
    got = gb.grouped_matmul(X.to(dev), W.to(dev), far.to(dev))
    want, size = grouped_want(X, W, offsets, identity, 1)
    oracle.close(got, want, oracle.product_bound(want, size, K + 1, dtype), "clamped")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_grouped_infinities_stay_in_their_group(dev, dtype):
    g = seeded("inf groups")
    offsets = torch.tensor([0, 20, 45], dtype=torch.int32)
    X, W = normal(g, 45, 40, dtype=dtype), normal(g, 2, 40, 48, dtype=dtype)
    X[44, 39] = NAN
    W[0, 39, 47] = INF
    say("inf groups", dtype)
    got = gb.grouped_matmul(X.to(dev), W.to(dev), offsets.to(dev)).cpu()
    assert got[44].isnan().all() and got[20:44].isfinite().all() and got[:20, :47].isfinite().all()
    assert not got[:20, 47].isfinite().any()


# --- weighted sums -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 8), (5, 8, 1000), (17, 4, 2048), (2, 3, 5001), (70, 1, 72), (4, 0, 9), (300, 6, 130)])
def test_combine_and_its_gradients(dev, dtype, pad, T, k, N):
    g = seeded("combine", T, k, N)
    P = T * k + 3
    position = torch.randperm(P, generator=g)[:T * k].int().reshape(T, k)
    if T * k > 2:
        position[0, 0], position[-1, -1] = -1, P + 9
    weight = normal(g, T, k)
    Y, dout = normal(g, P, N, dtype=dtype), normal(g, T, N, dtype=dtype)
    say("combine", T, k, N, pad, dtype)
    for w in (weight, None):
        ws = torch.ones(T, k, dtype=torch.float64) if w is None else weight.double()
        want, size = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
        dY_want, dw_want, dw_size = torch.full((P, N), 7.0, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                p = int(position[t, j])
                if 0 <= p < P:
                    want[t] += ws[t, j] * Y[p].double()
                    size[t] += (ws[t, j] * Y[p].double()).abs()
                    dY_want[p] = ws[t, j] * dout[t].double()
                    dw_want[t, j] = (Y[p].double() * dout[t].double()).sum()
                    dw_size[t, j] = (Y[p].double() * dout[t].double()).abs().sum()
        wd = None if w is None else w.to(dev)
        full = torch.full((T, N + pad), 7.0, dtype=dtype, device=dev)
        gb.combine(strided(Y, pad, dev), position.to(dev), wd, out=full[:, :N])
        oracle.close(full[:, :N], want, oracle.product_bound(want, size, k + 1, dtype), "out")
        assert (full[:, N:] == 7.0).all()
        full = torch.full((P, N + pad), 7.0, dtype=dtype, device=dev)
        dY, dw = gb.combine_grad(strided(dout, pad, dev), strided(Y, pad, dev), position.to(dev), wd, out=full[:, :N])
        # one product in binary32, rounded again to the type
        oracle.close(dY, dY_want, dY_want.abs() * (oracle.STEP[dtype] + 2.0 ** -23) + oracle.TINY[dtype], "dY")
        assert (full[:, N:] == 7.0).all()
        oracle.close(dw, dw_want, oracle.product_bound(dw_want, dw_size, N + 1, torch.float32), "dweight")


# --- adapters -----------------------------------------------------------------------
ADAPTERS = [
    # T, K, N, R, n
    (1, 1, 1, 1, 1), (1, 64, 128, 16, 3), (3, 130, 70, 5, 2), (16, 256, 264, 8, 40), (17, 200, 72, 24, 4), (64, 512, 256, 32, 64),
    (130, 96, 136, 33, 3), (300, 128, 200, 64, 5), (20, 64, 64, 200, 2), (50, 1000, 63, 4, 50), (5, 0, 8, 4, 2), (9, 40, 40, 0, 3),
    (33, 4096, 256, 16, 30), (515, 64, 200, 8, 4), (780, 130, 72, 40, 5), (560, 72, 330, 130, 2),
    (2060, 64, 200, 8, 4), (2055, 130, 72, 40, 5), (2049, 72, 330, 130, 2), (2051, 66, 1, 33, 2),
]


def adapters_want(X, W, A, B, adapter, scale):
    want = X.double() @ W.double()
    size = X.double().abs() @ W.double().abs()
    for t, a in enumerate(adapter.tolist()):
        if 0 <= a < A.shape[0]:
            low = X[t].double() @ A[a].double()
            want[t] += float(scale[a]) * (low @ B[a].double())
            size[t] += abs(float(scale[a])) * ((X[t].double().abs() @ A[a].double().abs()) @ B[a].double().abs())
    return want, size


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("runs", [False, True], ids=["mixed", "runs"])
@pytest.mark.parametrize("T,K,N,R,n", ADAPTERS)
def test_adapters(dev, dtype, pad, runs, T, K, N, R, n):
    g = seeded("adapters", T, K, N, R, n)
    X, W = normal(g, T, K, dtype=dtype), normal(g, K, N, dtype=dtype, scale=max(K, 1) ** -0.5)
    A, B = normal(g, n, K, R, dtype=dtype, scale=max(K, 1) ** -0.5), normal(g, n, R, N, dtype=dtype)
    adapter = torch.randint(-1, n + 1, (T,), generator=g, dtype=torch.int32)          # -1 and n: none
    if runs:
        adapter = adapter.sort().values
    scale = 0.5 + torch.rand(n, generator=g)
    say("adapters", T, K, N, R, n, pad, runs, dtype)
    want, size = adapters_want(X, W, A, B, adapter, scale)
    full = torch.full((T, N + pad), 7.0, dtype=dtype, device=dev)
    gb.adapter_matmul(strided(X, pad, dev), strided(W, pad, dev), strided(A, pad, dev), strided(B, pad, dev), adapter.to(dev),
                      scale.to(dev), out=full[:, :N])
    # the two low-rank sums follow one another; U is kept to 2^-16 (bf16: high + low parts) of its row's largest at least
    bound = oracle.product_bound(want, size, K + 2 * R + 4, dtype)
    low_top = torch.zeros(T, 1, dtype=torch.float64)
    for t, a in enumerate(adapter.tolist()):
        if 0 <= a < n and R:
            low_top[t] = float(scale[a]) * (X[t].double() @ A[a].double()).abs().max() * B[a].double().abs().sum(0).max()
    oracle.close(full[:, :N], want, bound + (0 if dtype == torch.float32 else 2.0 ** -16) * low_top, "Y")
    assert (full[:, N:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,N,R,n,run", [(2055, 4160, 8, 3, 700), (2100, 2300, 40, 60, 3), (4100, 4200, 16, 2, 4100)])
def test_adapters_large_tiles_whole_and_cut(dev, dtype, T, N, R, n, run):
    """Whole large tiles, cut ones, and the small ones behind them; `run` rows of an adapter side by side."""
    K = 40
    g = seeded("large adapters", T, N, R, n)
    X, W = normal(g, T, K, dtype=dtype).to(dev), normal(g, K, N, dtype=dtype).to(dev)
    A, B = normal(g, n, K, R, dtype=dtype, scale=K ** -0.5).to(dev), normal(g, n, R, N, dtype=dtype).to(dev)
    adapter = ((torch.arange(T) // run) % (n + 1) - 1).int()
    scale = 0.5 + torch.rand(n, generator=g)
    say("large adapters", T, N, R, n, dtype)
    got = gb.adapter_matmul(X, W, A, B, adapter.to(dev), scale.to(dev))
    want, size = torch.mm(X.double(), W.double()), torch.mm(X.double().abs(), W.double().abs())
    for a in range(n):
        mine = torch.nonzero(adapter == a).flatten().to(dev)
        s, x = float(scale[a]), X.double()[mine]
        want[mine] += s * torch.mm(torch.mm(x, A[a].double()), B[a].double())
        size[mine] += s * torch.mm(torch.mm(x.abs(), A[a].double().abs()), B[a].double().abs())
    # U is kept to 2^-16 of its row's largest at least: R terms of that, relative to the magnitudes' sum
    close_on_gpu(got, want, size * (1 + (0 if dtype == torch.float32 else R * 2.0 ** -16 / (2 * 2.0 ** -23 * (K + 2 * R + 4)))),
                 K + 2 * R + 4, "Y")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [3, 40, 150, 600, 2100])
def test_adapters_infinities_stay_with_their_requests(dev, dtype, T):
    g = seeded("inf adapters", T)
    X, W = normal(g, T, 64, dtype=dtype), normal(g, 64, 72, dtype=dtype)
    A, B = normal(g, 3, 64, 8, dtype=dtype), normal(g, 3, 8, 72, dtype=dtype)
    A[1, 5, 2], B[1, 3, 4] = INF, NAN
    adapter = (torch.arange(T) % 4 - 1).int()
    say("inf adapters", T, dtype)
    got = gb.adapter_matmul(X.to(dev), W.to(dev), A.to(dev), B.to(dev), adapter.to(dev)).cpu()
    assert got[adapter != 1].isfinite().all()
    assert not got[adapter == 1][:, 4].isfinite().any()
    want, size = adapters_want(X, W, A, B, torch.where(adapter == 1, -1, adapter), torch.ones(3))
    keep = adapter != 1
    oracle.close(got[keep], want[keep], (oracle.product_bound(want, size, 64 + 20, dtype) + 2.0 ** -12 * size)[keep], "others")


@pytest.mark.parametrize("factor", [2.0 ** -30, 2.0 ** 14])
@pytest.mark.parametrize("T", [20, 600, 2100])
def test_adapters_half_precision_range(dev, T, factor):
    """The low-rank intermediate may lie outside the 16-bit type's range."""
    g = seeded("range")
    X, W = normal(g, T, 64, dtype=torch.float16, scale=2.0 ** -3), normal(g, 64, 40, dtype=torch.float16)
    A, B = normal(g, 2, 64, 8, dtype=torch.float16), normal(g, 2, 8, 40, dtype=torch.float16, scale=2.0 ** -8)
    adapter = (torch.arange(T) % 2).int()
    scale = torch.tensor([factor, factor])
    say("half range", factor)
    W *= 0
    want, size = adapters_want(X, W, A, B, adapter, scale)
    got = gb.adapter_matmul(X.to(dev), W.to(dev), A.to(dev), B.to(dev), adapter.to(dev), scale.to(dev))
    oracle.close(got, want, oracle.product_bound(want, size, 64 + 20, torch.float16) + 2.0 ** -16 * size, "Y")


@pytest.mark.parametrize("T", [20, 600, 2100])
def test_adapters_half_precision_infinity_beside_large_values(dev, T):
    """X . A of +inf and of -120000, past the type's range: their sum is +inf."""
    X = torch.full((T, 2), 60000.0, dtype=torch.float16)
    A = torch.tensor([[INF, -1.0], [1.0, -1.0]], dtype=torch.float16)[None]
    B, W = torch.ones(1, 2, 24, dtype=torch.float16), torch.ones(2, 24, dtype=torch.float16)
    adapter = torch.full((T,), -1, dtype=torch.int32)
    adapter[5] = 0
    say("infinity beside large", T)
    got = gb.adapter_matmul((X * 2.0 ** -3).to(dev), W.to(dev), A.to(dev), B.to(dev), adapter.to(dev),
                            torch.tensor([8.0], device=dev)).cpu()
    assert (got[5] == INF).all()
    assert (got[adapter < 0] == 15000.0).all()       # 2 * 7500, exact


# --- together, as a layer uses them ----------------------------------------------------
def test_expert_layer_forward_and_backward(dev):
    """Router, map, two expert products with silu between, weighted sum; all gradients against 64-bit autograd."""
    T, E, k, K, N = 150, 6, 2, 64, 96
    g = seeded("layer")
    X, Wr = normal(g, T, K), normal(g, K, E, scale=K ** -0.5)
    W1, W2 = normal(g, E, K, N, scale=K ** -0.5), normal(g, E, N, K, scale=N ** -0.5)
    up = normal(g, T, K)
    Xd, Wrd, W1d, W2d, upd = (t.to(dev) for t in (X, Wr, W1, W2, up))

    logits = gb.matmul(Xd, Wrd)
    weight, index = gb.route(logits, k, normalize=True)
    offsets, order, position = gb.expert_map(index, E)
    h = gb.grouped_matmul(Xd, W1d, offsets, order=order, per_row=k)
    a = torch.nn.functional.silu(h)
    y = gb.grouped_matmul(a, W2d, offsets)
    out = gb.combine(y, position, weight)

    dy, dweight = gb.combine_grad(upd, y, position, weight)
    da = gb.grouped_grad_x(dy, W2d, offsets)
    dW2 = gb.grouped_grad_w(a, dy, offsets)
    s = torch.sigmoid(h)
    dh = da * s * (1 + h * (1 - s))
    dW1 = gb.grouped_grad_w(Xd, dh, offsets, order=order, per_row=k)
    dX = gb.combine(gb.grouped_grad_x(dh, W1d, offsets), position)
    dlogits = gb.route_grad(logits, index, dweight, normalize=True)
    dX = dX + gb.matmul(dlogits, Wrd.t().contiguous())
    dWr = gb.matmul(Xd.t().contiguous(), dlogits)

    leaves = [t.double().requires_grad_(True) for t in (X, Wr, W1, W2)]
    x, wr, w1, w2 = leaves
    at = index.cpu().long()
    w = oracle.route_weight_of(x @ wr, index.cpu(), "softmax", True, 1.0)
    rows = []
    for j in range(k):
        hj = torch.bmm(x.unsqueeze(1), w1[at[:, j]])
        rows.append(w[:, j:j + 1] * torch.bmm(torch.nn.functional.silu(hj), w2[at[:, j]]).squeeze(1))
    ref = rows[0] + rows[1]
    (ref * up.double()).sum().backward()
    # a chain of binary32 sums of some hundred terms of size about 1: relative to the largest element
    for name, got, want in (("out", out, ref.detach()), ("dX", dX, x.grad), ("dWr", dWr, wr.grad), ("dW1", dW1, w1.grad),
                            ("dW2", dW2, w2.grad)):
        oracle.close(got, want, 2.0 ** -23 * 1000 * want.abs().max(), name)


def test_layer_gradient_against_differences(dev):
    """The kernels' own forward pass, differenced along random directions of the expert weights."""
    T, E, k, K, N = 40, 4, 2, 32, 32
    g = seeded("differences")
    X, W, up = normal(g, T, K).to(dev), normal(g, E, K, N).to(dev), normal(g, T, N).to(dev)
    weight, index = gb.route(normal(g, T, E).to(dev), k, normalize=True)
    offsets, order, position = gb.expert_map(index, E)

    def value(w):
        y = gb.grouped_matmul(X, w, offsets, order=order, per_row=k)
        return float((gb.combine(y, position, weight).double() * up.double()).sum())
    y = gb.grouped_matmul(X, W, offsets, order=order, per_row=k)
    dy, _ = gb.combine_grad(up, y, position, weight)
    dW = gb.grouped_grad_w(X, dy, offsets, order=order, per_row=k)
    for trial in range(4):
        d = normal(g, E, K, N).to(dev)
        step = 0.5                                   # the value is linear in W: no truncation error
        diff = (value(W + step * d) - value(W - step * d)) / (2 * step)
        want = float((dW.double() * d.double()).sum())
        # T*N outputs of size under K, each off by under 2^-23 * 2K relative to sqrt(K): well under 1e-2 in all
        assert abs(diff - want) < 1e-2 + 1e-4 * abs(want)


def test_calls_on_another_stream_and_in_a_graph(dev):
    T, E, k, K, N, R = 70, 8, 2, 64, 72, 8
    g = seeded("stream")
    X, W = normal(g, T, K, dtype=torch.bfloat16).to(dev), normal(g, E, K, N, dtype=torch.bfloat16).to(dev)
    A, B = normal(g, 3, K, R, dtype=torch.bfloat16).to(dev), normal(g, 3, R, N, dtype=torch.bfloat16).to(dev)
    adapter = (torch.arange(T) % 4 - 1).int().to(dev)
    l = normal(g, T, E).to(dev)

    def everything(stream=None):
        weight, index = gb.route(l, k, normalize=True, stream=stream)
        offsets, order, position = gb.expert_map(index, E, stream=stream)
        y = gb.grouped_matmul(X, W, offsets, order=order, per_row=k, stream=stream)
        out = gb.combine(y, position, weight, stream=stream)
        dy, dw = gb.combine_grad(out, y, position, weight, stream=stream)
        dx = gb.grouped_grad_x(dy, W, offsets, stream=stream)
        dW = gb.grouped_grad_w(X, dy, offsets, order=order, per_row=k, stream=stream)
        dl = gb.route_grad(l, index, dw, normalize=True, stream=stream)
        z = gb.adapter_matmul(X, W[0], A, B, adapter, stream=stream)
        return [weight, index, offsets, order, position, y, out, dy, dw, dx, dW, dl, z]

    say("eager")
    want = [t.clone() for t in everything()]
    torch.cuda.synchronize()
    say("another stream")
    side = torch.cuda.Stream()
    for a, b in zip(want, everything(side)):
        side.synchronize()
        assert torch.equal(a, b)
    say("captured")
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = everything()
    for replay in range(3):
        l.copy_(normal(seeded("replay", replay), T, E).to(dev))
        graph.replay()
        torch.cuda.synchronize()
        mine = everything()
        torch.cuda.synchronize()
        for a, b in zip(mine, got):
            assert torch.equal(a, b)


def test_two_streams_at_once(dev):
    """Calls with workspaces of their own on two streams, many times, give what they give one after the other."""
    T, E, k, N, R = 300, 64, 8, 136, 16
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for q in range(2):
        g = seeded("streams", q)
        index = torch.randint(-1, E, (T * 500, k), generator=g, dtype=torch.int32).to(dev)
        X, W = normal(g, T, 256, dtype=torch.float16).to(dev), normal(g, 256, N, dtype=torch.float16).to(dev)
        A, B = normal(g, 5, 256, R, dtype=torch.float16).to(dev), normal(g, 5, R, N, dtype=torch.float16).to(dev)
        adapter = torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32).to(dev)
        sets.append((index, X, W, A, B, adapter))

    def both(index, X, W, A, B, adapter, stream=None):
        return [*gb.expert_map(index, E, stream=stream), gb.adapter_matmul(X, W, A, B, adapter, stream=stream)]

    say("one after the other")
    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    say("at once")
    got = [[], []]
    for _ in range(10):
        for q in range(2):
            got[q].append(both(*sets[q], stream=sides[q]))
    torch.cuda.synchronize()
    for q in range(2):
        for run in got[q]:
            for a, b in zip(run, want[q]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_offsets_past_the_places_are_clamped(dev, dtype):
    g = seeded("clamped", dtype)
    X, W = normal(g, 10, 24, dtype=dtype).to(dev), normal(g, 2, 24, 40, dtype=dtype).to(dev)
    dY = normal(g, 10, 40, dtype=dtype).to(dev)
    right = torch.tensor([0, 3, 10], dtype=torch.int32, device=dev)
    for wrong in ([-4, 3, 50], [0, 3, 2 ** 31 - 1], [-2 ** 31, 3, 11]):
        say("offsets", wrong, dtype)
        o = torch.tensor(wrong, dtype=torch.int32, device=dev)
        assert torch.equal(gb.grouped_matmul(X, W, o), gb.grouped_matmul(X, W, right))
        assert torch.equal(gb.grouped_grad_x(dY, W, o), gb.grouped_grad_x(dY, W, right))
        assert torch.equal(gb.grouped_grad_w(X, dY, o), gb.grouped_grad_w(X, dY, right))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("K", [57, 63, 64, 65, 71, 72, 73, 128, 136])
@pytest.mark.parametrize("N", [1, 2, 7])
def test_narrow_matrices_at_the_end_of_their_memory(dev, dtype, K, N):
    """Rows of a few elements, whose last chunks would span several rows; what follows is NaN."""
    g = seeded("narrow", K, N)
    ld = N + N % 2
    W = normal(g, 2, K, N, dtype=dtype)
    buf = torch.full((2 * K * ld + 64,), NAN, dtype=dtype, device=dev)
    Wd = buf[:2 * K * ld].view(2, K, ld)[:, :, :N]
    Wd.copy_(W.to(dev))
    X = normal(g, 40, K, dtype=dtype)
    offsets = torch.tensor([0, 17, 40], dtype=torch.int32)
    say("narrow", K, N, dtype)
    want, size = grouped_want(X, W, offsets, torch.arange(40, dtype=torch.int32), 1)
    got = gb.grouped_matmul(X.to(dev), Wd, offsets.to(dev))
    oracle.close(got, want, oracle.product_bound(want, size, K + 1, dtype), "Y")
    none = torch.full((40,), -1, dtype=torch.int32, device=dev)
    want, size = X.double() @ W[1].double(), X.double().abs() @ W[1].double().abs()
    A, B = torch.zeros(1, K, 4, dtype=dtype, device=dev), torch.zeros(1, 4, N, dtype=dtype, device=dev)
    got = gb.adapter_matmul(X.to(dev), Wd[1], A, B, none)
    oracle.close(got, want, oracle.product_bound(want, size, K + 1, dtype), "adapters")


def test_far_rows(dev):
    """Offsets past 2^32 bytes: rows far apart in one buffer."""
    ld = (1 << 31) // 64 + 8                                     # 33 rows span over 2^31 elements
    buf = torch.empty(66 * ld, dtype=torch.bfloat16, device=dev)
    X = buf.as_strided((66, 24), (ld, 1))
    g = seeded("far")
    x, W = normal(g, 66, 24, dtype=torch.bfloat16), normal(g, 2, 24, 40, dtype=torch.bfloat16)
    X.copy_(x.to(dev))
    offsets = torch.tensor([0, 5, 66], dtype=torch.int32)
    say("far rows")
    want, size = grouped_want(x, W, offsets, torch.arange(66, dtype=torch.int32), 1)
    got = gb.grouped_matmul(X, W.to(dev), offsets.to(dev))
    oracle.close(got, want, oracle.product_bound(want, size, 25, torch.bfloat16), "Y")
    got = gb.adapter_matmul(X, W[0].to(dev), torch.zeros(1, 24, 8, dtype=torch.bfloat16, device=dev),
                            torch.zeros(1, 8, 40, dtype=torch.bfloat16, device=dev), torch.zeros(66, dtype=torch.int32, device=dev))
    want, size = grouped_want(x, W[:1], torch.tensor([0, 66], dtype=torch.int32), torch.arange(66, dtype=torch.int32), 1)
    oracle.close(got, want, oracle.product_bound(want, size, 25, torch.bfloat16), "adapters")


def test_refusals_with_gpu_tensors(dev):
    x = torch.zeros(4, 8, device=dev)
    o = torch.zeros(3, dtype=torch.int32, device=dev)
    W = torch.zeros(2, 8, 5, device=dev)
    with pytest.raises(gb.GemmError) as e:
        gb.route(x, 9)
    assert e.value.status == gb.GEMM_F32_ERR_DIM
    with pytest.raises(ValueError):
        gb.route(x, 2, score="tanh")
    with pytest.raises(TypeError):
        gb.route(x, 2, bias=torch.zeros(8, dtype=torch.float64, device=dev))
    with pytest.raises(ValueError):
        gb.route(x, 2, bias=torch.zeros(7, device=dev))
    with pytest.raises(TypeError):
        gb.expert_map(torch.zeros(4, dtype=torch.int64, device=dev), 3)
    with pytest.raises(TypeError):
        gb.grouped_matmul(x, W.half(), o)
    with pytest.raises(ValueError):
        gb.grouped_matmul(x, W[:, :7], o)
    with pytest.raises(ValueError):
        gb.grouped_matmul(x, W.transpose(1, 2).contiguous().transpose(1, 2), o)
    with pytest.raises(ValueError):
        gb.grouped_matmul(x, W[:1].expand(2, 8, 5), o)
    with pytest.raises(TypeError):
        gb.grouped_matmul(x, W, o.cpu())
    with pytest.raises(ValueError):
        gb.combine(x, torch.zeros(4, 3, dtype=torch.int32, device=dev)[:, :2])
    with pytest.raises(gb.GemmError) as e:
        gb.adapter_matmul(x, W[0], torch.zeros(1, 8, 4, device=dev), torch.zeros(1, 4, 5, device=dev), o[:1].expand(4).contiguous(),
                          workspace=torch.zeros(8, dtype=torch.uint8, device=dev))
    assert e.value.status == gb.GEMM_F32_ERR_WORKSPACE


# T, N on both sides of the limit between few rows (binary32 intermediate) and many
ADAPTER_ROWS = [(20, 24), (2100, 24), (20, 16400)]


@pytest.mark.parametrize("T,N", ADAPTER_ROWS)
@pytest.mark.parametrize("low", [2.0 ** -27, 2.0 ** -31, 1.3e-6, 2.0 ** -13 * 1.7], ids=["2^-27", "2^-31", "1.3e-6", "1.7*2^-13"])
def test_adapters_half_precision_unlike_ranks(dev, T, N, low):
    """A rank far below its row's largest one counts where the largest meets zeros."""
    x = torch.tensor([1.0, low * 2.0 ** 12], dtype=torch.float32).half()
    X = x.expand(T, 2).contiguous()
    A = torch.tensor([[1.0, 0.0], [0.0, 2.0 ** -12]], dtype=torch.float16)[None]
    B = torch.zeros(1, 2, N, dtype=torch.float16)
    B[0, 1] = 32768.0
    adapter = torch.zeros(T, dtype=torch.int32)
    adapter[::3] = -1
    say("unlike ranks", T, N, low)
    got = gb.adapter_matmul(X.to(dev), torch.zeros(2, N, dtype=torch.float16, device=dev), A.to(dev), B.to(dev), adapter.to(dev))
    u = float(x[1]) * 2.0 ** -12                     # exact in binary32, as is its product with 2^15
    want = torch.where(adapter[:, None] == 0, torch.tensor(u * 32768.0, dtype=torch.float64), torch.zeros((), dtype=torch.float64)).expand(T, N)
    # x has 11 bits: U is exact in two parts as long as it is a multiple of 2^-39 of the row's largest, 1; the
    # sum is one product; one rounding to half
    assert u % 2.0 ** -39 == 0
    oracle.close(got, want, oracle.STEP[torch.float16] * want.abs() + oracle.TINY[torch.float16], "Y")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,N", ADAPTER_ROWS)
@pytest.mark.parametrize("R", [8, 40])
def test_adapters_infinite_scale(dev, dtype, T, N, R):
    """scale = inf times a sum without zeros is the infinity of the sum's sign, however many ranks pad a panel."""
    X = torch.ones(T, 8, dtype=dtype)
    A = torch.full((2, 8, R), 0.25, dtype=dtype)
    B = torch.ones(2, R, N, dtype=dtype)
    B[:, :, N // 2:] = -1.0
    adapter = (torch.arange(T) % 2).int()
    say("infinite scale", T, N, R, dtype)
    got = gb.adapter_matmul(X.to(dev), torch.zeros(8, N, dtype=dtype, device=dev), A.to(dev), B.to(dev), adapter.to(dev),
                            torch.tensor([INF, 3.0], device=dev)).cpu().double()
    assert (got[::2, :N // 2] == INF).all() and (got[::2, N // 2:] == -INF).all()
    assert (got[1::2, :N // 2] == 6.0 * R).all() and (got[1::2, N // 2:] == -6.0 * R).all()       # exact: R * 3 * 2


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,N", ADAPTER_ROWS)
def test_adapters_infinity_in_the_second_factor(dev, dtype, T, N):
    """An infinity of B times a rank that is no zero is an infinity of the rank's sign, not NaN."""
    g = seeded("inf of B", T, N)
    X, W = normal(g, T, 40, dtype=dtype), normal(g, 40, N, dtype=dtype, scale=40 ** -0.5)
    A, B = normal(g, 3, 40, 33, dtype=dtype, scale=40 ** -0.5), normal(g, 3, 33, N, dtype=dtype)
    adapter = (torch.arange(T) % 4 - 1).int()
    low = torch.mm(X.double(), A[1].double())
    B[1, 3, 5], B[1, 32, 9] = INF, -INF
    say("infinity of B", T, N, dtype)
    got = gb.adapter_matmul(X.to(dev), W.to(dev), A.to(dev), B.to(dev), adapter.to(dev)).cpu().double()
    mine = adapter == 1
    # 40 products whose magnitudes' sum is under 9.2 are off by under 2 * 41 * 2^-23 * 9.2 < 2^-13; no rank here is that near to zero
    assert low[mine][:, [3, 32]].abs().min() > 2.0 ** -13
    assert torch.equal(got[mine][:, 5], INF * low[mine][:, 3].sign())
    assert torch.equal(got[mine][:, 9], -INF * low[mine][:, 32].sign())
    others = torch.ones(T, N, dtype=torch.bool)
    others[mine] = torch.tensor([n not in (5, 9) for n in range(N)])
    assert got[others].isfinite().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N", ADAPTER_ROWS)
@pytest.mark.parametrize("x,a,b", [(1.0, 2.0 ** -20, 2.0 ** 127), (2.0 ** -66, 2.0 ** -60, 2.0 ** 127), (2.0 ** 63, 2.0 ** 63, 2.0 ** -120),
                                   (2.0 ** 100, 2.0 ** 10, 2.0 ** -100), (2.0 ** -30, 2.0 ** -30, 2.0 ** 100)])
def test_adapters_factors_far_from_one(dev, dtype, T, N, x, a, b):
    """Sums that the type holds although one of their factors is near its largest or smallest value."""
    X, A = torch.full((T, 1), x, dtype=dtype), torch.full((1, 1, 8), a, dtype=dtype)
    B = torch.full((1, 8, N), b, dtype=dtype)
    say("far from one", T, N, x, a, b, dtype)
    got = gb.adapter_matmul(X.to(dev), torch.zeros(1, N, dtype=dtype, device=dev), A.to(dev), B.to(dev),
                            torch.zeros(T, dtype=torch.int32, device=dev))
    assert (got.double() == 8.0 * x * a * b).all()   # powers of two: exact


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,R", [(2048, 16), (320, 17), (321, 64), (640, 64), (641, 20), (256, 65), (257, 65), (384, 130), (385, 256)])
def test_adapters_next_to_the_limits_of_few_rows(dev, dtype, T, R):
    K, N, n = 200, 136, 4
    g = seeded("row limits", T, R)
    X, W = normal(g, T, K, dtype=dtype), normal(g, K, N, dtype=dtype, scale=K ** -0.5)
    A, B = normal(g, n, K, R, dtype=dtype, scale=K ** -0.5), normal(g, n, R, N, dtype=dtype)
    adapter = torch.randint(-1, n + 1, (T,), generator=g, dtype=torch.int32)
    scale = 0.5 + torch.rand(n, generator=g)
    say("row limits", T, R, dtype)
    want, size = adapters_want(X, W, A, B, adapter, scale)
    got = gb.adapter_matmul(X.to(dev), W.to(dev), A.to(dev), B.to(dev), adapter.to(dev), scale.to(dev))
    # U is off by 2^-16 of itself, or 2^-22 of itself and 2^-39 of its row's largest, which 2^-16 of the magnitudes' sum covers:
    # the magnitudes of a row's ranks, sums of 200 terms, are alike
    oracle.close(got, want, oracle.product_bound(want, size, K + R + 4, dtype) + (0 if dtype == torch.float32 else 2.0 ** -16) * size, "Y")


def whole_numbers(g, *shape, dtype):
    """-2 .. 2: every partial sum of under 2^22 products is exact in binary32, so a result is the exact sum rounded once."""
    return torch.randint(-2, 3, shape, generator=g).to(dtype)


def takes_256(grad_w, G, P, M, N, cus):
    """The rule by which 16-bit products take tiles of 256 x 256."""
    rows = 2 * G * -(-M // 256) if grad_w else 2 * (P // 256) + min(G, P)
    return rows * -(-N // 256) * 5 >= 6 * cus


def pieces_of_the_last_round(tiles, cus):
    rest = tiles % cus
    return 4 if 4 * rest <= cus else 2 if 2 * rest <= cus else 1


GROUPS_256 = [1200, 0, 700, 1, 650]      # 12 row tiles of 256; one group longer than 1024 places, one empty


@pytest.mark.parametrize("dtype", TYPES[1:], ids=IDS[1:])
@pytest.mark.parametrize("pad", [0, 1], ids=["odd rows", "even rows"])       # staged loads, direct loads
@pytest.mark.parametrize("op,A,B,pieces,listed", [
    (*shape, listed) for shape in (
        ("forward", 333, 3579, 1), ("forward", 333, 5627, 4), ("forward", 72, 7165, 2),
        ("grad_x", 3579, 333, 1), ("grad_x", 5627, 333, 4), ("grad_x", 7165, 72, 2),
        ("grad_w", 1797, 2309, 1), ("grad_w", 1797, 1801, 4), ("grad_w", 1797, 2101, 2))
    for listed in (False, True) if not (listed and shape[0] == "grad_x")])      # that one knows no order
def test_grouped_tiles_of_256(dev, dtype, pad, op, A, B, pieces, listed):
    """Every product's largest tile, whole and with its last round cut: sums of whole numbers, equal."""
    K, N, G = A, B, len(GROUPS_256)
    g = seeded("256", op, K, N)
    offsets = torch.tensor([0] + GROUPS_256, dtype=torch.int32).cumsum(0).int()
    used = int(offsets[-1])
    P = used + 3                                     # three places in no group
    cus = torch.cuda.get_device_properties(dev).multi_processor_count
    row_tiles = sum(-(-n // 256) for n in GROUPS_256)
    M, C = (K, N) if op == "grad_w" else (0, N if op == "forward" else K)
    if cus == 256:
        assert takes_256(op == "grad_w", G, P, M, C, cus)
        tiles = (G * -(-M // 256) if op == "grad_w" else row_tiles) * -(-C // 256)
        assert pieces_of_the_last_round(tiles, cus) == pieces
    say("tiles of 256", op, K, N, pad, listed, dtype)
    rows = P if not listed else (P + 1) // 2
    order = torch.randperm(2 * rows, generator=g)[:P].int()
    if listed:
        order[7], order[used:] = -1, -1
    at = order.long().div(2, rounding_mode="floor").to(dev) if listed else torch.arange(P, device=dev)
    off = offsets.to(dev)
    list_ = dict(order=order.to(dev), per_row=2) if listed else {}

    def places_of(X):
        x = X.double()[at.clamp_min(0)]
        x[at < 0] = 0.0
        return x

    def check(got, want, what):
        assert torch.equal(got, want.to(dtype)), f"{what}: {int((got != want.to(dtype)).sum())} elements differ"
    if op != "grad_w":
        W = strided(whole_numbers(g, G, K, N, dtype=dtype), pad, dev)
        I = strided(whole_numbers(g, rows if op == "forward" else P, K if op == "forward" else N, dtype=dtype), pad, dev)
        full = torch.full((P, C + pad), 7.0, dtype=dtype, device=dev)
        if op == "forward":
            gb.grouped_matmul(I, W, off, out=full[:, :C], **list_)
        else:
            gb.grouped_grad_x(I, W, off, out=full[:, :C])
        x = places_of(I) if op == "forward" else I.double()
        for e in range(G):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            w = W[e].double() if op == "forward" else W[e].double().t().contiguous()
            check(full[lo:hi, :C], torch.mm(x[lo:hi], w), (op, e))
        assert (full[used:] == 7.0).all() and (full[:, C:] == 7.0).all()
    else:
        X = strided(whole_numbers(g, rows, K, dtype=dtype), pad, dev)
        dY = strided(whole_numbers(g, P, N, dtype=dtype), pad, dev)
        full = torch.full((G, K, N + pad), 7.0, dtype=dtype, device=dev)
        gb.grouped_grad_w(X, dY, off, out=full[:, :, :N], **list_)
        x = places_of(X)
        for e in range(G):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            check(full[e, :, :N], torch.mm(x[lo:hi].t().contiguous(), dY[lo:hi].double()), (op, e))
        assert (full[:, :, N:] == 7.0).all()


@pytest.mark.parametrize("rows,K,N", [(8, 4096, 512), (100, 4096, 72), (700, 4096, 200)])
def test_binary32_sums_are_no_single_long_chain(dev, rows, K, N):
    """Errors of binary32 products against 64 bits, in the root mean square.

    n additions in one chain of partial sums that grow like sqrt(k) for random signs are off by sqrt(sum over k of
    (2^-24 / sqrt(3))^2 k) = 2^-24 sqrt(n / 6) of the result's size sqrt(n).  The matrix cores add 4 products an
    instruction: 4096 k are 1024 additions, 2^-24 * 13 = 7.8e-7, with the instructions' own roundings more; parts of at
    most 512 + 32 k and 8 parts are 2^-24 * sqrt(136 / 6 + 8 / 6) = 2.9e-7 the same way.  The limit is between the two.
    """
    g = seeded("chains", rows, K, N)
    G = 8
    offsets = (torch.arange(G + 1) * rows).int()
    X, W = normal(g, G * rows, K).to(dev), normal(g, G, K, N).to(dev)
    dY = normal(g, G * rows, N).to(dev)
    say("chains", rows, K, N)

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())
    Y = gb.grouped_matmul(X, W, offsets.to(dev))
    want = torch.cat([torch.mm(X[e * rows:(e + 1) * rows].double(), W[e].double()) for e in range(G)])
    assert off(Y, want) < 5.5e-7
    # the other products, with K the summed index
    Wt = W.transpose(1, 2).contiguous()                         # [G, N, K]
    dX = gb.grouped_grad_x(X, Wt, offsets.to(dev))
    assert off(dX, want) < 5.5e-7
    long = torch.tensor([0, K], dtype=torch.int32, device=dev)
    A, B = X[:rows].t().contiguous(), W[0].contiguous()         # [K, rows], [K, N]
    dW = gb.grouped_grad_w(A, B, long)
    assert off(dW[0], torch.mm(A.t().double().contiguous(), B.double())) < 5.5e-7
    Z = gb.adapter_matmul(X.repeat(2, 1)[:600], W[0], torch.zeros(1, K, 33, device=dev), torch.zeros(1, 33, N, device=dev),
                          torch.full((min(600, 2 * G * rows),), -1, dtype=torch.int32, device=dev))
    assert off(Z, torch.mm(X.repeat(2, 1)[:600].double(), W[0].double())) < 5.5e-7
