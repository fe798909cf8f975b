"""The operators of a feed-forward block on the GPU against plain 64-bit
implementations (ffn_oracle.py).  8-bit rows and stored sums are equal; the
others are within the bounds worked out there."""
import math
import sys
import zlib

import pytest

from dense_fp32_gemm_amd import binding as gb
import ffn_oracle as oracle
import rows_oracle

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]
GATES = ["silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def say(*msg):
    print("[ffn]", *msg, file=sys.__stderr__, flush=True)


def seeded(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def strided(t, pad, dev, fill=NAN):
    """A copy on the GPU whose rows are `pad` elements further apart, filled around."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype)
    wide[..., :t.shape[-1]] = t
    return wide.to(dev)[..., :t.shape[-1]]


def put(t, dev):
    return None if t is None else t.to(dev)


# --- norm ---------------------------------------------------------------------------
# rows of one element to rows that do not fit the registers (a wave, 256 and 1024 threads a row)
NORMS = [(1, 1), (3, 7), (1, 64), (5, 100), (4, 512), (9, 513), (2, 1000), (7, 1024), (3, 2048), (5, 2050), (2, 4096), (3, 8192), (2, 8200),
         (1, 16384), (2, 16392), (1, 20000), (1500, 72), (1100, 600)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T,N", NORMS)
def test_rms_norm(dev, dtype, pad, T, N):
    g = seeded("norm", T, N)
    X, R, w = normal(g, T, N, dtype=dtype), normal(g, T, N, dtype=dtype, scale=2.0), 1 + normal(g, N, scale=0.2)
    X[T // 2] *= 30
    eps = 1e-5
    say("rms_norm", T, N, pad, dtype)
    for res, weight in ((R, w), (None, w), (R, None)):
        S = oracle.summed(X, res)
        want = oracle.normed(S, weight, eps)
        x, r = strided(X, pad, dev), None if res is None else strided(res, pad, dev)
        full = torch.full((T, N + pad), 7.0, dtype=dtype, device=dev)
        got = gb.rms_norm(x, put(weight, dev), eps=eps, residual=r, out=full[:, :N])
        if res is not None:
            got, s = got
            assert torch.equal(s.cpu(), S)
        # the row's factor and two products in binary32, then the type
        oracle.close(got, want, want.abs() * (4 * oracle.U + oracle.STEP[dtype]) + oracle.TINY[dtype], "Y")
        assert (full[:, N:] == 7.0).all()
        Q, scale, *more = gb.rms_norm_int8(x, put(weight, dev), eps=eps, residual=r)
        want_q, want_scale = oracle.int8_rows(want)
        assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)
        assert len(more) == (res is not None) and all(torch.equal(m.cpu(), S) for m in more)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("N", [40, 1500, 40000])
def test_rms_norm_in_place(dev, dtype, N):
    """The sum over the residual or X, the norm over X."""
    g = seeded("in place", N)
    X, R = normal(g, 5, N, dtype=dtype), normal(g, 5, N, dtype=dtype)
    S = oracle.summed(X, R)
    want, alone = oracle.normed(S, None, 1e-6), oracle.normed(X, None, 1e-6)
    room = 4 * oracle.U + oracle.STEP[dtype]
    say("in place", N, dtype)
    x, r = X.to(dev), R.to(dev)
    y, s = gb.rms_norm(x, residual=r, out_sum=r, out=x)
    assert y is x and s is r and torch.equal(r.cpu(), S)
    oracle.close(x, want, want.abs() * room + oracle.TINY[dtype], "over X")
    x, r = X.to(dev), R.to(dev)
    Q, scale, s = gb.rms_norm_int8(x, residual=r, out_sum=x)
    assert torch.equal(x.cpu(), S) and torch.equal(Q.cpu(), oracle.int8_rows(want)[0])
    x = X.to(dev)
    gb.rms_norm(x, out=x)
    oracle.close(x, alone, alone.abs() * room + oracle.TINY[dtype], "alone")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("N", [24, 1500, 40000])
def test_rms_norm_rows_of_every_kind(dev, dtype, N):
    """Zeros, the largest and smallest numbers, infinities and NaN, each in a row of its own."""
    g = seeded("kinds", N)
    X = normal(g, 10, N, dtype=dtype)
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    X[1] = 0
    X[2] = big
    X[3] = small
    X[4] = 0
    X[4, N // 2] = small * torch.finfo(dtype).eps                # the smallest number there is
    X[5, 3] = INF
    X[6, N - 1] = NAN
    X[7, 0] = big
    X[8, 1::2] = 0
    w = 1 + normal(g, N, scale=0.1)
    w[2] = 0
    say("kinds", N, dtype)
    want = oracle.normed(X, w, 1e-6)
    got = gb.rms_norm(X.to(dev), w.to(dev))
    # products with numbers under binary32's normal ones: half of its smallest number, times the next factor
    oracle.close(got, want, want.abs() * (4 * oracle.U + oracle.STEP[dtype]) + oracle.TINY[dtype] + 2.0 ** -148, "Y")
    Q, scale = gb.rms_norm_int8(X.to(dev), w.to(dev))
    want_q, want_scale = oracle.int8_rows(want)
    assert scale.cpu().isnan().tolist() == want_scale.isnan().tolist() == [t in (5, 6) for t in range(10)]
    assert torch.equal(scale.cpu().nan_to_num(), want_scale.nan_to_num()) and torch.equal(Q.cpu(), want_q)
    w[5] = NAN                                                   # a weight reaches every row
    Q, scale = gb.rms_norm_int8(X.to(dev), w.to(dev))
    assert scale.isnan().all() and not Q.any()
    w[5] = INF
    Q, scale = gb.rms_norm_int8(X.to(dev), w.to(dev))
    bad = oracle.int8_rows(oracle.normed(X, w, 1e-6))[1].isnan()
    assert torch.equal(scale.isnan().cpu(), bad) and not Q[bad].any()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("T,N", NORMS + [(5000, 200), (2500, 2100), (300, 17000)])
def test_rms_norm_grad(dev, dtype, pad, T, N):
    g = seeded("norm grad", T, N)
    S, d, ds, w = normal(g, T, N, dtype=dtype), normal(g, T, N, dtype=dtype), normal(g, T, N, dtype=dtype), 1 + normal(g, N, scale=0.2)
    S[T // 3] *= 50
    say("rms_norm_grad", T, N, pad, dtype)
    for extra, weight in ((ds, w), (None, None)):
        dX, dw, bound, size = oracle.norm_grad(d, S, weight, 1e-5, extra)
        full = torch.full((T, N + pad), 7.0, dtype=dtype, device=dev)
        got, got_w = gb.rms_norm_grad(strided(d, pad, dev), strided(S, pad, dev), put(weight, dev), eps=1e-5,
                                      dsum=None if extra is None else strided(extra, pad, dev), out=full[:, :N])
        oracle.close(got, dX, bound, "dX")
        assert (full[:, N:] == 7.0).all()
        # a workgroup adds its rows one by one in binary32 (there are at least as many workgroups as compute units
        # or rows), each term off by two half steps; the workgroups' sums in binary64
        chain = -(-T // torch.cuda.get_device_properties(dev).multi_processor_count)
        oracle.close(got_w, dw, (chain + 4) * oracle.U * size + 2.0 ** -149, "dweight")


def test_rms_norm_grad_in_place_and_repeatable(dev):
    g = seeded("grad in place")
    S, d, ds, w = (normal(g, *s, dtype=torch.bfloat16).to(dev) for s in ((700, 1000), (700, 1000), (700, 1000), (1000,)))
    w = w.float()
    dX, dw = gb.rms_norm_grad(d, S, w, dsum=ds)
    for which in range(3):
        ins = [d.clone(), S.clone(), ds.clone()]
        got, got_w = gb.rms_norm_grad(ins[0], ins[1], w, dsum=ins[2], out=ins[which])
        assert got is ins[which] and torch.equal(got, dX) and torch.equal(got_w, dw)


def test_rms_norm_of_no_rows_and_no_columns(dev):
    assert gb.rms_norm(torch.zeros(0, 8, device=dev)).shape == (0, 8)
    assert gb.rms_norm(torch.zeros(3, 0, device=dev)).shape == (3, 0)
    Q, scale = gb.rms_norm_int8(torch.zeros(3, 0, device=dev))
    assert Q.shape == (3, 0) and scale.tolist() == [2.0 ** -126] * 3
    dX, dw = gb.rms_norm_grad(torch.zeros(0, 8, device=dev), torch.zeros(0, 8, device=dev))
    assert dX.shape == (0, 8) and dw.tolist() == [0.0] * 8
    assert gb.quantize(torch.zeros(0, 8, device=dev))[0].shape == (0, 8)


# --- rows in 8 bits -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T,N", NORMS)
def test_quantize(dev, dtype, pad, T, N):
    g = seeded("quantize", T, N)
    X = normal(g, T, N, dtype=dtype)
    X[T // 2] *= 100
    say("quantize", T, N, pad, dtype)
    Q, scale = gb.quantize(strided(X, pad, dev))
    want_q, want_scale = oracle.int8_rows(X.double())
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("top", [127.0, 254.0, 190.5, 31.75])
def test_quantize_values_on_rounding_borders(dev, dtype, top):
    """Rows of halves of their scale: ties go to the even number."""
    s = top / 127
    X = torch.cat([torch.tensor([top]), (torch.arange(-254, 255) / 2) * s]).repeat(3, 1).to(dtype)
    Q, scale = gb.quantize(X.to(dev))
    want_q, want_scale = oracle.int8_rows(X.double())
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)
    if dtype == torch.float32:
        assert Q[0, 1:].cpu().tolist() == [round(i / 2) for i in range(-254, 255)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("pad", [0, 2, 8])
@pytest.mark.parametrize("T,N", [(1, 1), (3, 7), (5, 100), (2, 512), (9, 513), (3, 2048), (2, 4100), (3, 8192), (2, 16392), (600, 96)])
def test_quantize_gated(dev, dtype, kind, pad, T, N):
    g = seeded("quantize gated", T, N)
    X = normal(g, T, 2 * N, dtype=dtype, scale=2.0)
    X[T // 2, :N] -= 6                                           # the gate's left side
    say("quantize", kind, T, N, pad, dtype)
    Q, scale = gb.quantize(strided(X, pad, dev), gate=kind)
    want_q, want_scale = oracle.int8_rows(oracle.gate(X[:, :N].double(), kind) * X[:, N:].double())
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)


@pytest.mark.parametrize("kind", [None] + GATES)
@pytest.mark.parametrize("N", [12, 1500, 40000])
def test_quantize_rows_of_every_kind(dev, kind, N):
    g = seeded("quantize kinds", N)
    X = normal(g, 12, N if kind is None else 2 * N)
    X[1] = 0
    X[2] = torch.finfo(torch.float32).max
    X[3, 2] = INF
    X[4, N - 1] = NAN
    X[5] *= 2.0 ** -130                                          # scales at their smallest
    X[6] *= 2.0 ** -149
    X[7, :N] = -1000.0                                           # silu(-1000) is 0 in 64 bits too
    X[8, :N] = -85.0                                             # under binary32's numbers, times large ones
    X[8, N:] = 1e38
    X[9, :N] = -11.0
    X[10] *= 2.0 ** 120
    X[11, ::2] = 0
    say("quantize kinds", kind, N)
    Q, scale = gb.quantize(X.to(dev), gate=kind)
    y = X.double() if kind is None else oracle.gate(X[:, :N].double(), kind) * X[:, N:].double()
    want_q, want_scale = oracle.int8_rows(y)
    assert torch.equal(scale.cpu().isnan(), want_scale.isnan()) and torch.equal(scale.cpu().nan_to_num(), want_scale.nan_to_num())
    assert torch.equal(Q.cpu(), want_q)


# Factors that are no normal binary32 numbers (and keep few of their digits there) times large ones: the product's
# rounding shows every digit that was lost.
@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("N", [24, 1500, 4096, 40000])
def test_quantize_small_gates_of_large_numbers(dev, dtype, kind, N):
    g = seeded("small gates", N)
    X = normal(g, 9, 2 * N)
    for t, (gate, other) in enumerate([(-140, 60), (-134, 60), (-138, 60), (-141, 60), (-130, 60), (-128, 50), (-124, 40), (-145, 120)]):
        X[t, :N] *= 2.0 ** gate
        X[t, N:] *= 2.0 ** other
    X[1, :N:3] = 0.0
    # 1.5 of the smallest number (2 if rounded) times 2^100, beside 1.7 of an ordinary gate: the row's largest is the other
    X[8] = 0.0
    X[8, 1], X[8, N + 1], X[8, N - 2], X[8, 2 * N - 2] = 3 * 2.0 ** -149, 2.0 ** 100, 20.0, 1.7 * 2.0 ** -49 / 20
    X = X.to(dtype)
    say("small gates", kind, N, dtype)
    Q, scale = gb.quantize(X.to(dev), gate=kind)
    want_q, want_scale = oracle.int8_rows(oracle.gate(X[:, :N].double(), kind) * X[:, N:].double())
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)


@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("N", [24, 1500, 4096, 40000])
def test_rms_norm_int8_small_elements_of_large_weights(dev, dtype, N):
    """One element of each row sets its root mean square; the others, under binary32's normal numbers after it, set its scale."""
    g = seeded("large weights", N)
    X, w = normal(g, 5, N), (1 + normal(g, N, scale=0.2)) * 2.0 ** 60
    for t, small in enumerate((-36, -40, -42, -44, -30)):
        X[t] *= 2.0 ** small
    X[:, N // 2] = 2.0 ** 100
    w[N // 2] = 2.0 ** -88
    X = X.to(dtype)
    say("large weights", N, dtype)
    Q, scale = gb.rms_norm_int8(X.to(dev), w.to(dev))
    want_q, want_scale = oracle.int8_rows(oracle.normed(X, w, 1e-6))
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)


@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("by", [60, -60])
@pytest.mark.parametrize("N", [24, 4096, 40000])
def test_rms_norm_int8_products_beyond_binary32(dev, dtype, by, N):
    """S times its weight passes binary32's ends on either side, and the row's factor brings it back."""
    g = seeded("far products", N, by)
    X, w = normal(g, 6, N), (1 + normal(g, N, scale=0.2)) * 2.0 ** by
    for t, size in enumerate((80, 100, 66, -60, -70, -80)):
        X[t] *= 2.0 ** size
    X = X.to(dtype)
    say("far products", by, N, dtype)
    Q, scale = gb.rms_norm_int8(X.to(dev), w.to(dev), eps=2.0 ** -120)
    want_q, want_scale = oracle.int8_rows(oracle.normed(X, w, 2.0 ** -120))
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(Q.cpu(), want_q)


# --- 8-bit product -----------------------------------------------------------------------
def eight(g, T, K):
    return torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)


# few rows (1 to 48), tiles of 32 x 64, 64 x 64 and 64 x 128, and of 256 x 256 whole and cut
INT8 = [(1, 1, 1), (1, 16, 16), (2, 17, 15), (7, 65, 100), (16, 300, 256), (16, 4200, 513), (17, 4200, 70), (17, 33, 257), (48, 40, 90), (49, 40, 90), (32, 64, 2048), (33, 40, 1000), (64, 130, 4100),
        (520, 2050, 70), (1100, 2100, 96), (65, 1, 1), (65, 64, 128), (100, 129, 130), (129, 200, 1000), (300, 513, 77), (70, 300, 0), (3, 20, 0), (2000, 130, 64)]


def check_int8(dev, g, T, N, K, pad, dtype, with_bias):
    Q, W = eight(g, T, K), eight(g, N, K)
    s, ws = torch.rand(T, generator=g) * 0.1 + 0.001, torch.rand(N, generator=g) * 0.01 + 1e-4
    bias = normal(g, N) if with_bias else None
    want, bound = oracle.int8_product(Q, s, W, ws, bias, dtype)
    full = torch.full((T, N + pad), 7.0, dtype=dtype, device=dev)
    got = gb.int8_matmul(strided(Q, pad, dev, 99), s.to(dev), strided(W, pad, dev, -77), ws.to(dev), bias=put(bias, dev), out=full[:, :N])
    oracle.close(got, want, bound, "Y")
    assert (full[:, N:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 4, 16])
@pytest.mark.parametrize("T,N,K", INT8)
def test_int8_matmul(dev, dtype, pad, T, N, K):
    say("int8", T, N, K, pad, dtype)
    check_int8(dev, seeded("int8", T, N, K), T, N, K, pad, dtype, pad != 4)


@pytest.mark.parametrize("pad", [0, 1], ids=["direct loads", "staged loads"])
@pytest.mark.parametrize("T,N,K", [(4096, 4096, 128), (4200, 4100, 200), (2600, 5200, 300), (4096, 4864, 96), (8200, 2100, 144), (2600, 2600, 130)])
def test_int8_large_tiles_whole_and_cut(dev, pad, T, N, K):
    say("int8 large", T, N, K, pad)
    check_int8(dev, seeded("int8 large", T, N, K), T, N, K, pad, torch.bfloat16, False)


# More panels of 128 k than twice a ring has, the last one partial: 32 x 64 (four in the ring), 64 x 64 (four), 64 x 128
# (three), 256 x 256 whole (two) with a last round cut in four (four), and cut in two (three).
DEEP_INT8 = [(100, 130, 2100), (520, 2050, 1400), (1100, 2100, 1100), (4200, 4100, 1300), (2600, 2600, 1300)]


@pytest.mark.parametrize("pad", [0, 1, 4], ids=["rows as long as they are", "staged loads", "direct loads"])
@pytest.mark.parametrize("T,N,K", DEEP_INT8)
def test_int8_panels_in_turn(dev, pad, T, N, K):
    """Sums of many panels, exact: whole numbers under 2^24, every k a part of each (no element is 0)."""
    g = seeded("int8 deep", T, N, K)
    Q, W = (torch.where(x < 0, x, x + 1) for x in (torch.randint(-64, 64, s, generator=g, dtype=torch.int8) for s in ((T, K), (N, K))))
    say("int8 panels", T, N, K, pad)
    got = gb.int8_matmul(strided(Q, pad, dev, 99), torch.ones(T, device=dev), strided(W, pad, dev, -77), torch.ones(N, device=dev),
                         dtype=torch.float32)
    assert torch.equal(got.cpu(), (Q.double() @ W.double().t()).float())


@pytest.mark.parametrize("T", [3, 40, 100])
def test_int8_sums_are_exact_at_the_largest_depth(dev, T):
    """-128 times -128, 131071 of them: just inside 32 bits; one less in one place."""
    K = gb.GEMM_F32_MAX_INT8_DEPTH
    Q, W = torch.full((T, K), -128, dtype=torch.int8), torch.full((17, K), -128, dtype=torch.int8)
    W[3, K - 1] = -127
    W[4] = 127
    say("deep", T)
    one = torch.ones(T, device=dev), torch.ones(17, device=dev)
    got = gb.int8_matmul(Q.to(dev), one[0], W.to(dev), one[1], dtype=torch.float32).double().cpu()
    want = (Q.double() @ W.double().t()).float().double()          # one rounding to binary32
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [5, 80, 300])
@pytest.mark.parametrize("with_bias", [False, True])
def test_int8_results_in_binary32_are_rounded_once(dev, T, with_bias):
    """Scales from 2^-126 to 2^100, whose products no binary32 number may hold: sums of 0 stay 0, the others half a step off."""
    K, N = 200, 130
    g = seeded("int8 once", T)
    Q, W = eight(g, T, K), eight(g, N, K)
    Q[1] = 0
    s, ws = torch.rand(T, generator=g) + 0.5, torch.rand(N, generator=g) + 0.5
    for t, by in enumerate((0, 100, -126, -100, 100)):
        s[t::5] *= 2.0 ** by
    for n, by in enumerate((0, 100, -126, -40, -10, -30, 20)):
        ws[n::7] *= 2.0 ** by
    bias = normal(g, N) if with_bias else None
    say("int8 once", T, with_bias)
    got = gb.int8_matmul(Q.to(dev), s.to(dev), W.to(dev), ws.to(dev), bias=put(bias, dev), dtype=torch.float32)
    want = (Q.double() @ W.double().t()) * (s.double()[:, None] * ws.double())
    if with_bias:
        want = want + bias.double()
    want = torch.where(want.float().isinf(), want.float().double(), want)
    # half a step of binary32, and of binary64 before
    oracle.close(got, want, want.abs().nan_to_num(posinf=0) * (oracle.U + 2.0 ** -52) + 2.0 ** -150, "Y")


@pytest.mark.parametrize("T", [5, 80])
def test_int8_scales_that_are_not_finite_stay_in_their_row(dev, T):
    g = seeded("int8 nan", T)
    Q, W = eight(g, T, 64).to(dev), eight(g, 40, 64).to(dev)
    s, ws = torch.ones(T, device=dev), torch.ones(40, device=dev)
    plain = gb.int8_matmul(Q, s, W, ws)
    s[2] = NAN
    got = gb.int8_matmul(Q, s, W, ws)
    assert got[2].isnan().all() and torch.equal(got[:2], plain[:2]) and torch.equal(got[3:], plain[3:])


# --- gated projections --------------------------------------------------------------------
def places(g, T, k, E, drop=0.0):
    """offsets, order, position of a random choice, some slots left out, some experts without any."""
    score = torch.rand(T, E, generator=g)
    score[:, E // 2] = -1.0
    index = torch.topk(score, k, dim=1).indices.int()
    index[torch.rand(T, k, generator=g) < drop] = -1
    return rows_oracle.expert_map(index, E)


def check_gated(dev, dtype, pad, X, W, offsets, order, k, kind, save=True):
    """H and pre of every place, and that the places of no group are left alone."""
    G, N = W.shape[0], W.shape[2] // 2
    P = X.shape[0] if order is None else len(order)
    rows = X.double() if order is None else rows_oracle.rows_of(X, order, k)
    bounds = [0, P] if offsets is None else offsets.tolist()
    full = torch.full((P, N + pad), 7.0, dtype=dtype, device=dev)
    got = gb.gated_matmul(strided(X, pad, dev), strided(W, pad, dev), put(offsets, dev), order=put(order, dev), per_row=k, gate=kind,
                          save=save, out=full[:, :N])
    H, pre = got if save else (got, None)
    for e in range(G):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        want, bound, want_pre, bound_pre = oracle.gated(rows[lo:hi], W[e], kind, dtype)
        oracle.close(H[lo:hi], want, bound, "H")
        if save:
            oracle.close(pre[lo:hi], want_pre, bound_pre, "pre")
    assert (full[bounds[-1]:] == 7.0).all() and (full[:, N:] == 7.0).all()


SHAPES = [
    # T, E, k, K, N
    (1, 1, 1, 1, 1), (1, 4, 2, 8, 8), (5, 3, 1, 17, 33), (3, 8, 4, 64, 128), (40, 4, 2, 65, 63), (33, 70, 2, 96, 72),
    (200, 3, 2, 129, 100), (300, 2, 2, 72, 256), (260, 5, 3, 256, 24), (9, 2, 1, 0, 5), (513, 2, 1, 128, 66), (700, 130, 2, 64, 32),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T,E,k,K,N", SHAPES)
def test_gated_by_expert(dev, dtype, pad, T, E, k, K, N):
    g = seeded("gated", T, E, k, K, N)
    offsets, order, _ = places(g, T, k, E, drop=0.1)
    X, W = normal(g, T, K, dtype=dtype), normal(g, E, K, 2 * N, dtype=dtype, scale=max(K, 1) ** -0.5)
    say("gated", T, E, k, K, N, pad, dtype)
    check_gated(dev, dtype, pad, X, W, offsets, order, k, GATES[(T + pad) % 3])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (17, 100, 51), (33, 64, 96), (100, 130, 200), (400, 72, 130), (2, 2000, 40)])
def test_gated_dense(dev, dtype, kind, T, K, N):
    g = seeded("dense", T, K, N)
    X, W = normal(g, T, K, dtype=dtype), normal(g, 1, K, 2 * N, dtype=dtype, scale=2 * K ** -0.5)
    say("gated dense", T, K, N, kind, dtype)
    check_gated(dev, dtype, 0, X, W, None, None, 1, kind, save=T % 2 == 1)


@pytest.mark.parametrize("dtype", TYPES[1:], ids=IDS[1:])
@pytest.mark.parametrize("pad", [0, 1], ids=["direct loads", "staged loads"])
@pytest.mark.parametrize("T,E,k,K,N", [(4096, 1, 1, 96, 2048), (4200, 1, 1, 70, 2100), (2000, 2, 2, 64, 2200), (2300, 4, 2, 72, 1300), (4100, 1, 1, 64, 2300),
                                       (520, 1, 1, 200, 2200), (300, 2, 2, 64, 2200)])
def test_gated_large_tiles_whole_and_cut(dev, dtype, pad, T, E, k, K, N):
    g = seeded("gated large", T, E, k, K, N)
    offsets, order, _ = places(g, T, k, E) if E > 1 else (None, None, None)
    X, W = normal(g, T, K, dtype=dtype), normal(g, E, K, 2 * N, dtype=dtype, scale=K ** -0.5)
    say("gated large", T, E, k, K, N, pad, dtype)
    check_gated(dev, dtype, pad, X, W, offsets, order, k, "silu")


# More panels than twice a ring has, the last one partial.  16-bit types (64 k a panel): 32 x 64 (a ring of four), 64 x 128
# (three), 256 x 256 cut in four (four), in two (three), whole (two); binary32 (32 k): 32 x 64 and 64 x 64, whose sums
# are folded every 512 k.
DEEP_GATED = [(20, 40, 1100), (200, 200, 900), (520, 2200, 700), (1000, 2200, 650), (4200, 2100, 650)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 1], ids=["direct loads", "staged loads"])
@pytest.mark.parametrize("T,N,K", DEEP_GATED + [(300, 100, 1700)])
def test_gated_panels_in_turn(dev, dtype, pad, T, N, K):
    """Sums of many panels, exact: whole numbers, every k a part of each (no element is 0)."""
    if dtype == torch.float32:
        T, N = min(T, 500), min(N, 300)
    g = seeded("gated deep", T, N, K)
    X, W = (torch.tensor([-2.0, -1.0, 1.0, 2.0])[torch.randint(4, s, generator=g)].to(dtype) for s in ((T, K), (1, K, 2 * N)))
    say("gated panels", T, N, K, pad, dtype)
    H, pre = gb.gated_matmul(strided(X, pad, dev), strided(W, pad, dev), save=True)
    sums = X.double() @ W[0].double()
    assert torch.equal(pre.cpu(), sums.to(dtype))
    want = oracle.gate(sums[:, :N], "silu") * sums[:, N:]
    # (half: from 65520 on, half a step past its largest number, infinities)
    want = torch.where(want.to(dtype).isinf(), want.to(dtype).double(), want)
    err = (oracle.GATE_ERROR["silu"] + 2 * oracle.U) * want.abs() + oracle.LOST_VALUE * (1 + sums[:, N:].abs())
    oracle.close(H, want, err + oracle.STEP[dtype] * (want.abs() + err) + oracle.TINY[dtype], "H")


@pytest.mark.parametrize("dtype", TYPES[1:], ids=IDS[1:])
@pytest.mark.parametrize("bounds", [[0, 6100], [0, 2500, 6100], [5, 2000, 2000, 5900], [0, 700, 6100]])
def test_tiles_of_long_and_short_groups(dev, dtype, bounds):
    """256 x 256 tiles of groups of up to 24 row tiles, in bands and in whole columns, each once: whole numbers, exact."""
    G, P, K, N = len(bounds) - 1, 6100, 70, 1800
    g = seeded("bands", bounds)
    few = torch.tensor([-2.0, -1.0, 1.0, 2.0])
    X, W = (few[torch.randint(4, s, generator=g)].to(dtype) for s in ((P, K), (G, K, N)))
    off = None if bounds == [0, P] else torch.tensor(bounds, dtype=torch.int32, device=dev)
    say("bands", bounds, dtype)
    x, w = X.to(dev), W.to(dev)
    Y = gb.grouped_matmul(x, w, off, out=torch.full((P, N), 7.0, dtype=dtype, device=dev))
    pre = gb.gated_matmul(x, w, off, save=True)[1]
    # the gradient of X has K columns: the products' roles changed about
    dX = gb.grouped_grad_x(x, w.transpose(1, 2).contiguous(), off, out=torch.full((P, N), 7.0, dtype=dtype, device=dev))
    for e in range(G):
        lo, hi = bounds[e], bounds[e + 1]
        want = (X[lo:hi].double() @ W[e].double()).to(dtype)
        assert torch.equal(Y[lo:hi].cpu(), want) and torch.equal(pre[lo:hi].cpu(), want) and torch.equal(dX[lo:hi].cpu(), want)
    for out in (Y, dX):
        assert (out[:bounds[0]] == 7.0).all() and (out[bounds[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows", [3, 40, 300])
def test_gated_infinities_stay_in_their_places(dev, dtype, rows):
    """A NaN in a column of the gate, in one of the others and in a row of X reach what they meet alone."""
    g = seeded("gated nan", rows)
    X, W = normal(g, rows, 48, dtype=dtype), normal(g, 2, 48, 2 * 40, dtype=dtype)
    offsets = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=dev)
    plain = gb.gated_matmul(X.to(dev), W.to(dev), offsets)
    W[0, 7, 3] = NAN
    W[1, 9, 40 + 39] = NAN
    X[rows - 1, 5] = NAN
    got = gb.gated_matmul(X.to(dev), W.to(dev), offsets)
    bad = torch.zeros(rows, 40, dtype=torch.bool)
    bad[:rows // 2, 3] = True
    bad[rows // 2:, 39] = True
    bad[rows - 1] = True
    assert torch.equal(got.isnan().cpu(), bad)
    assert torch.equal(got.cpu()[~bad], plain.cpu()[~bad])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("P,N", [(1, 1), (3, 7), (5, 64), (2, 1000), (70, 72), (3, 2048), (2, 5001), (1000, 40)])
def test_gate_grad(dev, dtype, kind, pad, P, N):
    g = seeded("gate grad", P, N)
    pre, dH = normal(g, P, 2 * N, dtype=dtype, scale=3.0), normal(g, P, N, dtype=dtype)
    pre[P // 2, 0] = -300.0                                      # far on both sides
    pre[P // 2, N // 2] = 1000.0
    want, bound = oracle.gate_grad(dH, pre, kind)
    full = torch.full((P, 2 * N + pad), 7.0, dtype=dtype, device=dev)
    say("gate_grad", kind, P, N, pad, dtype)
    p = strided(pre, pad, dev)
    oracle.close(gb.gate_grad(strided(dH, pad, dev), p, gate=kind, out=full[:, :2 * N]), want, bound, "dpre")
    assert (full[:, 2 * N:] == 7.0).all()
    gb.gate_grad(dH.to(dev), p, gate=kind, out=p)
    assert torch.equal(p, full[:, :2 * N])


@pytest.mark.parametrize("kind", GATES)
def test_gates_and_slopes_to_a_few_steps(dev, kind):
    """act(g) and act'(g) in binary32, where nothing underflows, to the half steps that their steps leave.

    The exponential: its argument's part under binary32 is made up for; 2^x as the hardware gives it 2 half steps, the
    factor, their product 1 each: 4.  The reciprocal 2.
      silu       exponential, 1 + e, reciprocal, g s: 8.  Slope s (1 + g (1 - s)): s 7, 1 - s 7, sum and product 2: 16
      gelu       g^2 / 2 is off by a half step of itself, the exponential by g^2 / 2 half steps for that; t = 1 / (1 + 0.4 z):
                 constant, sum, reciprocal 4, which counts up to 1.6 times; the polynomial 6 (whose fit is 1); three products:
                 under 24 with the exponential's 4, and g^2 / 2.  Slope p + g e^(-g^2 / 2) / sqrt(2 pi): the same
      gelu_tanh  v = g (kA + kB g^2): two constants and three steps, 5 |v| half steps of the exponential; else as silu, 10.
                 Slope s + g s (1 - s) v': s and 1 - s each so, and six steps: 24 + 10 |v|
    """
    g = torch.linspace(-9, 12, 400001)
    n = g.numel()
    pre = torch.cat([g, torch.ones(n)])[None]
    got = gb.gate_grad(torch.ones(1, n, device=dev), pre.to(dev), gate=kind).cpu().double()[0]
    x = g.double()
    p, q = oracle.gate_parts(x, kind)
    v = math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3)
    value, slope = {"silu": (8.0, 16.0), "gelu": (24 + x * x, 24 + x * x), "gelu_tanh": (10 + 5 * v.abs(), 24 + 10 * v.abs())}[kind]
    oracle.close(got[n:], x * p, oracle.U * value * (x * p).abs(), "value")
    oracle.close(got[:n], p + q, oracle.U * (slope + 1) * (p.abs() + q.abs()), "slope")


@pytest.mark.parametrize("kind", GATES)
def test_gate_grad_of_the_largest_numbers(dev, kind):
    """Gates at the type's ends give the slopes 0 and 1, not NaN."""
    big = torch.finfo(torch.float32).max
    pre = torch.tensor([[big, -big, 1e20, -1e20, 2.0, 3.0, 4.0, 5.0]], device=dev)
    got = gb.gate_grad(torch.ones(1, 4, device=dev), pre, gate=kind).cpu()
    assert got.tolist() == [[2.0, 0.0, 4.0, 0.0, pre[0, 0].item(), 0.0, pre[0, 2].item(), 0.0]]


# --- together -----------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 30, 200])
def test_an_8_bit_block_as_it_is_served(dev, T):
    """norm -> 8 bits -> gate and up -> gate -> 8 bits -> down, each step's output the next one's input."""
    D, N = 192, 320
    g = seeded("served", T)
    X, R, w = normal(g, T, D, dtype=torch.bfloat16), normal(g, T, D, dtype=torch.bfloat16), 1 + normal(g, D, scale=0.1)
    Wu, Wd = normal(g, 2 * N, D, scale=D ** -0.5), normal(g, D, N, scale=N ** -0.5)
    say("served", T)
    wu, su = gb.quantize(Wu.to(dev))
    wd, sd = gb.quantize(Wd.to(dev))
    Q, s, S = gb.rms_norm_int8(X.to(dev), w.to(dev), residual=R.to(dev))
    pair = gb.int8_matmul(Q, s, wu, su)
    q2, s2 = gb.quantize(pair, gate="silu")
    Y = gb.int8_matmul(q2, s2, wd, sd)

    oq, os_ = oracle.int8_rows(oracle.normed(oracle.summed(X, R), w, 1e-6))
    assert torch.equal(Q.cpu(), oq) and torch.equal(s.cpu(), os_)
    ou, osu = oracle.int8_rows(Wu.double())
    want, bound = oracle.int8_product(oq, os_, ou, osu, None, torch.bfloat16)
    oracle.close(pair, want, bound, "pair")
    p = pair.cpu().double()
    oq, os_ = oracle.int8_rows(oracle.gate(p[:, :N], "silu") * p[:, N:])
    assert torch.equal(q2.cpu(), oq) and torch.equal(s2.cpu(), os_)
    od, osd = oracle.int8_rows(Wd.double())
    want, bound = oracle.int8_product(oq, os_, od, osd, None, torch.bfloat16)
    oracle.close(Y, want, bound, "Y")
    # the whole against the same block in 64 bits: 8 bits leave each row a relative error (2-norm) of at most
    # sqrt(N) / 2 of 127 steps of its largest element, here about a hundredth, three times over
    n = oracle.normed(oracle.summed(X, R), w, 1e-6)
    f = n @ Wu.double().t()
    exact = (oracle.gate(f[:, :N], "silu") * f[:, N:]) @ Wd.double().t()
    assert (Y.cpu().double() - exact).norm() < 0.1 * exact.norm()


def block(X, R, w, W, Wd, kind):
    """A dense block in 64 bits, differentiable."""
    S = X + R
    n = S * torch.rsqrt((S * S).mean(1, keepdim=True) + 1e-6) * w
    N = W.shape[1] // 2
    f = n @ W
    return S + (oracle.gate(f[:, :N], kind) * f[:, N:]) @ Wd


@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("T,D,N", [(1, 24, 40), (37, 65, 51), (150, 128, 200)])
def test_a_dense_block_and_its_gradients(dev, kind, T, D, N):
    """norm with residual, gated pair, down-projection, and back, against autograd in 64 bits and against differences."""
    g = seeded("block", T, D, N)
    X, R, w = normal(g, T, D), normal(g, T, D), 1 + normal(g, D, scale=0.1)
    W, Wd, dY = normal(g, D, 2 * N, scale=D ** -0.5), normal(g, N, D, scale=N ** -0.5), normal(g, T, D)
    say("block", T, D, N, kind)
    x, r, wn, w1, w2, dy = (t.to(dev) for t in (X, R, w, W, Wd, dY))
    n, S = gb.rms_norm(x, wn, residual=r)
    H, pre = gb.gated_matmul(n, w1[None], gate=kind, save=True)
    Y = S + gb.grouped_matmul(H, w2[None])
    dH = gb.grouped_grad_x(dy, w2[None])
    dWd = gb.grouped_grad_w(H, dy)[0]
    dpre = gb.gate_grad(dH, pre, gate=kind)
    dn = gb.grouped_grad_x(dpre, w1[None])
    dW = gb.grouped_grad_w(n, dpre)[0]
    dX, dw = gb.rms_norm_grad(dn, S, wn, dsum=dy)

    leaves = [t.double().requires_grad_(True) for t in (X, R, w, W, Wd)]
    out = block(*leaves, kind)
    (out * dY.double()).sum().backward()
    # a chain of binary32 steps: each output is a sum of under 1000 terms of size about 1, each off by a few dozen
    # half steps: 2^-24 * 64 of the largest, and the terms' errors add up like their square root
    def near(got, want, what):
        assert (got.double().cpu() - want).norm() <= 64 * oracle.U * want.norm(), what
    near(Y, out.detach(), "Y")
    for got, leaf, what in ((dX, leaves[0], "dX"), (dX, leaves[1], "dR"), (dw, leaves[2], "dw"), (dW, leaves[3], "dW"), (dWd, leaves[4], "dWd")):
        near(got, leaf.grad, what)
    # along a random direction of all leaves, by differences in 64 bits
    with torch.no_grad():
        move = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in leaves]
        h = 1e-5
        ahead, behind = (sum_ for sum_ in ((block(*(t + e * h * m for t, m in zip(leaves, move)), kind) * dY.double()).sum() for e in (1, -1)))
        got = sum((d.double().cpu() * m).sum() for d, m in zip((dX, dX, dw, dW, dWd), move))
        size = sum((d.double().cpu() * m).abs().sum() for d, m in zip((dX, dX, dw, dW, dWd), move))
        assert abs((ahead - behind) / (2 * h) - got) <= 1e-6 * size


def test_expert_block_forward_and_backward(dev):
    """route -> slot map -> gated experts -> down -> weighted sum, and the gradient back to the tokens."""
    T, E, k, D, N = 90, 6, 2, 64, 48
    g = seeded("experts")
    X, logits = normal(g, T, D), normal(g, T, E)
    W, Wd, dout = normal(g, E, D, 2 * N, scale=D ** -0.5), normal(g, E, N, D, scale=N ** -0.5), normal(g, T, D)
    x, w1, w2, do = (t.to(dev) for t in (X, W, Wd, dout))
    weight, index = gb.route(logits.to(dev), k, normalize=True)
    offsets, order, position = gb.expert_map(index, E)
    H, pre = gb.gated_matmul(x, w1, offsets, order=order, per_row=k, save=True)
    Y = gb.grouped_matmul(H, w2, offsets)
    out = gb.combine(Y, position, weight)
    dY, dweight = gb.combine_grad(do, Y, position, weight)
    dWd = gb.grouped_grad_w(H, dY, offsets)
    dpre = gb.gate_grad(gb.grouped_grad_x(dY, w2, offsets), pre)
    dW = gb.grouped_grad_w(x, dpre, offsets, order=order, per_row=k)
    dX = gb.combine(gb.grouped_grad_x(dpre, w1, offsets), position)

    leaves = [t.double().requires_grad_(True) for t in (X, W, Wd)]
    want = torch.zeros(T, D, dtype=torch.float64)
    wt, ix = weight.cpu().double(), index.cpu()
    for e in range(E):
        for j in range(k):
            mine = torch.nonzero(ix[:, j] == e).flatten()
            f = leaves[0][mine] @ leaves[1][e]
            y = (oracle.gate(f[:, :N], "silu") * f[:, N:]) @ leaves[2][e]
            want = want.index_add(0, mine, wt[mine, j, None] * y)
    (want * dout.double()).sum().backward()
    for got, ref in ((out, want.detach()), (dX, leaves[0].grad), (dW, leaves[1].grad), (dWd, leaves[2].grad)):
        assert (got.double().cpu() - ref).norm() <= 64 * oracle.U * ref.norm()


# --- streams, graphs, far rows, refusals -------------------------------------------------------
def everything(a):
    """One call of each operator; outputs in a list."""
    y, s = gb.rms_norm(a["x"], a["w"], residual=a["r"])
    q, qs, s2 = gb.rms_norm_int8(a["x"], a["w"], residual=a["r"])
    pair = gb.int8_matmul(q, qs, a["w8"], a["s8"], bias=a["b"])
    q2, qs2 = gb.quantize(pair, gate="gelu_tanh")
    few = gb.int8_matmul(q[:5], qs[:5], a["w8"], a["s8"], dtype=torch.float32)
    h, pre = gb.gated_matmul(a["x"], a["W"], a["offsets"], order=a["order"], per_row=2, save=True)
    dpre = gb.gate_grad(h, pre)
    dx, dw = gb.rms_norm_grad(y, s, a["w"], dsum=a["r"])
    dense = gb.gated_matmul(a["x"], a["W"][:1], gate="gelu")
    back = gb.grouped_grad_x(dense.repeat(1, 2), a["W"][:1])
    grad = gb.grouped_grad_w(a["x"], dense.repeat(1, 2))
    return [y, s, q, qs, s2, pair, q2, qs2, few, h, pre, dpre, dx, dw, dense, back, grad]


def inputs(dev, seed):
    g = seeded("everything", seed)
    T, D, N = 100, 136, 72
    offsets, order, _ = places(g, T, 2, 5)
    a = dict(x=normal(g, T, D, dtype=torch.bfloat16), r=normal(g, T, D, dtype=torch.bfloat16), w=1 + normal(g, D, scale=0.1),
             w8=eight(g, 2 * N, D), s8=torch.rand(2 * N, generator=g) * 0.01, b=normal(g, 2 * N),
             W=normal(g, 5, D, 2 * N, dtype=torch.bfloat16, scale=D ** -0.5), offsets=offsets, order=order)
    return {k: v.to(dev) for k, v in a.items()}


def test_calls_on_another_stream_and_in_a_graph(dev):
    a, b = inputs(dev, 1), inputs(dev, 2)
    want_a, want_b = everything(a), everything(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything(a)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want_a))
    held = {k: v.clone() for k, v in a.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything(held)
    say("captured")
    for turn, (src, want) in enumerate([(a, want_a), (b, want_b), (a, want_a), (b, want_b)]):
        for k in held:
            held[k].copy_(src[k])
        everything(a)                                            # the program's own work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        say("replayed", turn)
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_the_stream_argument(dev):
    a = inputs(dev, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = gb.rms_norm(a["x"], a["w"], stream=side)
    q, s = gb.quantize(a["x"], stream=side)
    z = gb.int8_matmul(a["w8"], a["s8"], a["w8"], a["s8"], stream=side)
    h, pre = gb.gated_matmul(a["x"], a["W"][:1], save=True, stream=side)
    d = gb.gate_grad(h, pre, stream=side)
    dx, dw = gb.rms_norm_grad(a["x"], a["x"], stream=side)
    q8 = gb.rms_norm_int8(a["x"], stream=side)
    side.synchronize()
    h2, pre2 = gb.gated_matmul(a["x"], a["W"][:1], save=True)
    for got, want in ((y, gb.rms_norm(a["x"], a["w"])), (q, gb.quantize(a["x"])[0]), (z, gb.int8_matmul(a["w8"], a["s8"], a["w8"], a["s8"])),
                      (h, h2), (pre, pre2), (d, gb.gate_grad(h2, pre2)), (dw, gb.rms_norm_grad(a["x"], a["x"])[1]), (q8[0], gb.rms_norm_int8(a["x"])[0])):
        assert torch.equal(got, want)


def test_two_streams_at_once(dev):
    ins = [inputs(dev, s) for s in (4, 5)]
    want = [everything(a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for turn in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = everything(ins[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_operands_that_start_on_odd_elements(dev, dtype):
    """Bases one element past an aligned address, and operands of unlike strides, give what aligned ones give."""
    g = seeded("odd base")
    T, N = 70, 96

    def shifted(t):
        wide = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev)[1:]
        return wide.view(t.shape).copy_(t)

    X, R, D = (normal(g, T, N, dtype=dtype).to(dev) for _ in range(3))
    P = normal(g, T, 2 * N, dtype=dtype).to(dev)
    w = shifted(1 + normal(g, N, scale=0.1).to(dev))
    far = strided(R.cpu(), 8, dev)
    for got, want in ((gb.rms_norm(shifted(X), w, residual=far), gb.rms_norm(X, w.clone(), residual=R)),
                      (gb.rms_norm_int8(X, w, residual=shifted(R)), gb.rms_norm_int8(X, w.clone(), residual=R)),
                      (gb.rms_norm_grad(shifted(D), X, w, dsum=far), gb.rms_norm_grad(D, X, w, dsum=R)),
                      (gb.quantize(shifted(P), gate="silu"), gb.quantize(P, gate="silu")), (gb.quantize(shifted(X)), gb.quantize(X))):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # (a product may be rounded to the type from binary32, or, by a mixed instruction, from its exact value: equal
    # only to within the bound, which counts both roundings)
    oracle.close(gb.gate_grad(shifted(D), P), *oracle.gate_grad(D.cpu(), P.cpu(), "silu"), "dpre")
    q, k = eight(g, T, N).to(dev), eight(g, 40, N).to(dev)
    s, ks = torch.rand(T, device=dev), torch.rand(40, device=dev)
    for rows in (5, T):
        want = gb.int8_matmul(q[:rows], s[:rows], k, ks, dtype=dtype)
        assert torch.equal(gb.int8_matmul(shifted(q[:rows]), s[:rows], shifted(k), shifted(ks), dtype=dtype), want)
        out = torch.empty(rows * 40 + 1, dtype=dtype, device=dev)[1:].view(rows, 40)
        assert torch.equal(gb.int8_matmul(q[:rows], s[:rows], k, ks, out=out), want)
    W = normal(g, 1, N, 80, dtype=dtype, scale=0.1).to(dev)
    want, bound, _, _ = oracle.gated(X.cpu().double(), W[0].cpu(), "silu", dtype)
    oracle.close(gb.gated_matmul(shifted(X), shifted(W)), want, bound, "H")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_many_short_rows(dev, dtype):
    """More rows than workgroups take at once, against the formulas in 64 bits on the GPU."""
    T, N = 100003, 24
    g = torch.Generator(device=dev).manual_seed(9)
    X = torch.randn(T, 2 * N, generator=g, device=dev).to(dtype)
    D = torch.randn(T, N, generator=g, device=dev).to(dtype)
    x = X[:, :N].contiguous()
    say("many rows", dtype)
    s = x.double()
    r = (s.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    oracle.close(gb.rms_norm(x), (s * r).cpu(), (s * r).cpu().abs() * (4 * oracle.U + oracle.STEP[dtype]) + oracle.TINY[dtype], "Y")
    dX, dw, bound, size = oracle.norm_grad(D.cpu(), x.cpu(), None, 1e-6, None)
    got, got_w = gb.rms_norm_grad(D, x)
    oracle.close(got, dX, bound, "dX")
    oracle.close(got_w, dw, (T // 256 + 5) * oracle.U * size, "dweight")
    for (Q, scale), y in ((gb.quantize(x), s), (gb.rms_norm_int8(x), s * r),
                          (gb.quantize(X, gate="gelu"), oracle.gate(s, "gelu") * X[:, N:].double())):
        want = (y.abs().amax(1) / 127).float().clamp_min(2.0 ** -126)
        assert torch.equal(scale, want) and torch.equal(Q, torch.round(y / want.double()[:, None]).to(torch.int8))
    want, bound = oracle.gate_grad(D.cpu(), X.cpu(), "silu")
    oracle.close(gb.gate_grad(D, X), want, bound, "dpre")


# Rows of several waves, more of them than the device's workgroups take at once (eight of 256 threads a compute unit): a
# workgroup's second row meets the LDS slots that its first one used.
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("chunks,threads", [(138, 128), (263, 256), (520, 512), (1030, 1024), (2060, 1024)])
def test_second_rows_of_several_waves(dev, dtype, chunks, threads):
    N = chunks * 16 // torch.finfo(dtype).bits * 8
    T = torch.cuda.get_device_properties(dev).multi_processor_count * 8 * 256 // threads * 9 // 8 + 3
    g = torch.Generator(device=dev).manual_seed(chunks)
    X = torch.randn(T, 2 * N, generator=g, device=dev)
    X *= 2.0 ** (torch.arange(T, device=dev) % 7 - 3)[:, None]           # unlike rows side by side
    X = X.to(dtype)
    x, R = X[:, :N].contiguous(), X[:, N:].contiguous()
    w = 1 + torch.randn(N, generator=g, device=dev) * 0.2
    say("second rows", T, N, dtype)
    S = (x.double() + R.double()).to(dtype)
    s = S.double()
    want = s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w.double()
    got, sum_ = gb.rms_norm(x, w, eps=1e-5, residual=R)
    assert torch.equal(sum_, S)
    room = want.abs() * (4 * oracle.U + oracle.STEP[dtype]) + oracle.TINY[dtype]
    assert ((got.double() - want).abs() <= room).all()
    for (Q, scale), y in ((gb.rms_norm_int8(x, w, eps=1e-5, residual=R)[:2], want), (gb.quantize(x), x.double()),
                          (gb.quantize(X, gate="silu"), oracle.gate(x.double(), "silu") * R.double()),
                          (gb.quantize(X, gate="gelu_tanh"), oracle.gate(x.double(), "gelu_tanh") * R.double())):
        top = (y.abs().amax(1) / 127).float()
        assert torch.equal(scale, top) and torch.equal(Q, torch.round(y / top.double()[:, None]).to(torch.int8))


def test_far_rows(dev):
    """Rows whose offsets pass 2^31 elements."""
    ld = (1 << 30) + 64
    g = seeded("far")
    small = normal(g, 4, 40, dtype=torch.bfloat16)
    wide = torch.empty(3 * ld + 64, dtype=torch.bfloat16, device=dev).as_strided((4, 64), (ld, 1))
    far = wide[:, :40]
    far.copy_(small)
    near = small.to(dev)
    say("far rows")
    assert torch.equal(gb.rms_norm(far), gb.rms_norm(near))
    for x, y in zip(gb.quantize(far) + gb.rms_norm_int8(far, residual=far) + gb.rms_norm_grad(far, far, dsum=far),
                    gb.quantize(near) + gb.rms_norm_int8(near, residual=near) + gb.rms_norm_grad(near, near, dsum=near)):
        assert torch.equal(x, y)
    assert torch.equal(gb.gate_grad(far[:, :20], far), gb.gate_grad(near[:, :20], near))
    W = normal(g, 1, 40, 24, dtype=torch.bfloat16).to(dev)
    H = gb.gated_matmul(near, W)
    assert torch.equal(gb.gated_matmul(far, W, out=wide[:, 48:60]), H)
    q = eight(g, 4, 40).to(dev)
    far8 = torch.empty(3 * ld + 40, dtype=torch.int8, device=dev).as_strided((4, 40), (ld, 1))
    far8.copy_(q)
    one = torch.ones(4, device=dev)
    assert torch.equal(gb.int8_matmul(far8, one, far8, one), gb.int8_matmul(q, one, q, one))
    many = eight(g, 80, 40).to(dev)
    assert torch.equal(gb.int8_matmul(many, torch.ones(80, device=dev), far8, one), gb.int8_matmul(many, torch.ones(80, device=dev), q, one))


def test_refusals_with_gpu_tensors(dev):
    x, q = torch.zeros(4, 8, device=dev), torch.zeros(4, 8, dtype=torch.int8, device=dev)
    s, w = torch.ones(4, device=dev), torch.ones(8, device=dev)
    with pytest.raises(gb.GemmError):
        gb.rms_norm(x, eps=0.0)
    with pytest.raises(TypeError):
        gb.rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        gb.rms_norm(x, w[:7])
    with pytest.raises(ValueError):
        gb.rms_norm(x, out_sum=x)
    with pytest.raises(TypeError):
        gb.rms_norm(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        gb.rms_norm(x, residual=x[:3])
    with pytest.raises(ValueError):
        gb.rms_norm(x.t(), torch.ones(4, device=dev))
    with pytest.raises(ValueError):
        gb.rms_norm_grad(x, x[:, :7])
    with pytest.raises(ValueError, match="even"):
        gb.quantize(x[:, :7], gate="silu")
    with pytest.raises(ValueError, match="gate"):
        gb.quantize(x, gate="relu")
    with pytest.raises(TypeError):
        gb.int8_matmul(x, s, q, s)
    with pytest.raises(TypeError):
        gb.int8_matmul(q, s, q.to(torch.uint8), s)
    with pytest.raises(ValueError):
        gb.int8_matmul(q, s, q[:, :7], s)
    with pytest.raises(ValueError):
        gb.int8_matmul(q, s[:3], q, s)
    with pytest.raises(TypeError):
        gb.int8_matmul(q, s, q, s, dtype=torch.float64)
    with pytest.raises(TypeError):
        gb.int8_matmul(q, s, q, s, dtype=torch.bfloat16, out=x[:, :4])
    with pytest.raises(TypeError):
        gb.int8_matmul(q, s.cpu(), q, s)
    deep = torch.zeros(1, gb.GEMM_F32_MAX_INT8_DEPTH + 1, dtype=torch.int8, device=dev)
    with pytest.raises(gb.GemmError):
        gb.int8_matmul(deep, s[:1], deep, s[:1])
    W = torch.zeros(1, 8, 6, device=dev)
    with pytest.raises(ValueError, match="even"):
        gb.gated_matmul(x, W[:, :, :5])
    with pytest.raises(ValueError):
        gb.gated_matmul(x, W.repeat(2, 1, 1))
    with pytest.raises(ValueError):
        gb.gated_matmul(x, torch.zeros(1, 7, 6, device=dev))
    with pytest.raises(ValueError, match="gate"):
        gb.gated_matmul(x, W, gate=None)
    with pytest.raises(gb.GemmError):
        gb.gated_matmul(x, W, order=torch.zeros(4, dtype=torch.int32, device=dev), per_row=0)
    with pytest.raises(ValueError):
        gb.gate_grad(x, x)
