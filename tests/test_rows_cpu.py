"""CPU checks of the row-chosen products: refusals, workspace sizes, the
declared ABI, and the oracle's own gradients against differences."""
import os
import re

import pytest

from dense_fp32_gemm_amd import binding as gb
import rows_oracle as oracle

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f32_rows.h")
FAKE = 0x100000


def test_library_exports_and_binds_every_declared_function():
    names = sorted(set(re.findall(r"GEMM_F32_API\s+[\w\s\*]*?\b(gemm_f32\w*)\s*\(", open(HEADER).read())))
    assert len(names) == 11, names
    for n in names:
        assert hasattr(gb.load(), n) and hasattr(gb, n), n


def test_constants_match_the_header():
    found = re.findall(r"#define (GEMM_F32_(?:TYPE|SCORE|MAX)_\w+)\s+(\d+)", open(HEADER).read())
    assert len(found) == 8
    for name, value in found:
        assert getattr(gb, name) == int(value), name


ROUTE = dict(type=0, T=4, E=8, k=2, logits=FAKE, ldl=8, bias=0, score=0, groups=1, keep_groups=1, group_top=1,
             normalize=0, scale=1.0, weight=FAKE, index=FAKE)


@pytest.mark.parametrize("change,rc", [
    (dict(type=3), "TYPE"), (dict(type=-1), "TYPE"), (dict(T=-1), "DIM"), (dict(E=0), "DIM"), (dict(E=1025, ldl=1025), "DIM"),
    (dict(k=0), "DIM"), (dict(k=9), "DIM"), (dict(E=128, ldl=128, k=65), "DIM"), (dict(ldl=7), "LD"), (dict(score=2), "OPTION"),
    (dict(groups=0), "OPTION"), (dict(groups=3), "OPTION"), (dict(groups=2, keep_groups=3), "OPTION"),
    (dict(keep_groups=0), "OPTION"), (dict(group_top=0), "OPTION"), (dict(group_top=3), "OPTION"),
    (dict(E=130, ldl=130, groups=65), "OPTION"), (dict(logits=0), "NULL"), (dict(weight=0), "NULL"), (dict(index=0), "NULL"),
    (dict(logits=FAKE + 2), "ALIGN"), (dict(type=1, logits=FAKE + 1), "ALIGN"), (dict(bias=FAKE + 2), "ALIGN"),
    (dict(weight=FAKE + 1), "ALIGN"), (dict(T=0, logits=0, weight=0, index=0), None)])
def test_route_refuses(change, rc):
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_route(**{**ROUTE, **change}) == want


GRAD = dict(type=0, T=4, E=8, k=2, logits=FAKE, ldl=8, score=0, normalize=0, scale=1.0, index=FAKE, dweight=FAKE,
            dlogits=FAKE, lddl=8)


@pytest.mark.parametrize("change,rc", [
    (dict(type=3), "TYPE"), (dict(k=0), "DIM"), (dict(ldl=7), "LD"), (dict(lddl=7), "LD"), (dict(score=-1), "OPTION"),
    (dict(index=0), "NULL"), (dict(dlogits=0), "NULL"), (dict(dweight=FAKE + 2), "ALIGN"), (dict(T=0, logits=0), None)])
def test_route_grad_refuses(change, rc):
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_route_grad(**{**GRAD, **change}) == want


@pytest.mark.parametrize("change,rc", [
    (dict(S=-1), "DIM"), (dict(E=0), "DIM"), (dict(E=1025), "DIM"), (dict(offsets=0), "NULL"), (dict(index=0), "NULL"),
    (dict(position=0), "NULL"), (dict(order=FAKE + 2), "ALIGN"), (dict(S=200000), "WORKSPACE"),
    (dict(S=200000, workspace=FAKE, workspace_bytes=16), "WORKSPACE"),
    (dict(S=200000, workspace=FAKE + 4, workspace_bytes=1 << 30), "WORKSPACE")])
def test_expert_map_refuses(change, rc):
    base = dict(S=10, E=4, index=FAKE, offsets=FAKE, order=FAKE, position=FAKE)
    assert gb.gemm_f32_expert_map(**{**base, **change}) == getattr(gb, "GEMM_F32_ERR_" + rc)


def test_expert_map_workspace_only_for_many_slots():
    assert gb.gemm_f32_expert_map_ws_size(0, 8) == gb.gemm_f32_expert_map_ws_size(1 << 15, 1024) == 0
    assert gb.gemm_f32_expert_map_ws_size((1 << 15) + 1, 8) > 0
    assert gb.gemm_f32_expert_map_ws_size(-1, 8) == gb.gemm_f32_expert_map_ws_size(9, 0) == 0


GROUPED = dict(type=1, G=2, P=4, N=8, K=16, offsets=FAKE, order=FAKE, per_row=2, rows=2, X=FAKE, ldx=16, W=FAKE, ldw=8,
               stride_w=128, Y=FAKE, ldy=8)


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(G=-1), "DIM"), (dict(P=-1), "DIM"), (dict(N=-1), "DIM"), (dict(K=-1), "DIM"),
    (dict(rows=-1), "DIM"), (dict(order=0), "DIM"), (dict(ldx=15), "LD"), (dict(ldw=7), "LD"), (dict(ldy=7), "LD"),
    (dict(stride_w=127), "LD"), (dict(per_row=0), "OPTION"), (dict(offsets=0), "NULL"), (dict(X=0), "NULL"),
    (dict(W=0), "NULL"), (dict(Y=0), "NULL"), (dict(X=FAKE + 1), "ALIGN"), (dict(order=FAKE + 2), "ALIGN"),
    (dict(P=1 << 30, N=1 << 20, ldw=1 << 20, ldy=1 << 20, stride_w=1 << 24), "DIM"),
    (dict(G=0, offsets=0, Y=0), None), (dict(P=0, Y=0), None), (dict(N=0, Y=0, W=0), None)])
def test_grouped_refuses(change, rc):
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_grouped(**{**GROUPED, **change}) == want


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(P=-1), "DIM"), (dict(lddy=7), "LD"), (dict(lddx=15), "LD"), (dict(stride_w=1), "LD"),
    (dict(dY=0), "NULL"), (dict(dX=0), "NULL"), (dict(dX=FAKE + 1), "ALIGN"), (dict(K=0, dX=0), None)])
def test_grouped_grad_x_refuses(change, rc):
    base = dict(type=1, G=2, P=4, N=8, K=16, offsets=FAKE, dY=FAKE, lddy=8, W=FAKE, ldw=8, stride_w=128, dX=FAKE, lddx=16)
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_grouped_grad_x(**{**base, **change}) == want


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(K=-1), "DIM"), (dict(order=0), "DIM"), (dict(ldx=15), "LD"), (dict(lddw=7), "LD"),
    (dict(stride_dw=1), "LD"), (dict(per_row=-1), "OPTION"), (dict(dW=0), "NULL"), (dict(dY=0), "NULL"),
    (dict(dW=FAKE + 1), "ALIGN"), (dict(G=0, dW=0), None)])
def test_grouped_grad_w_refuses(change, rc):
    base = dict(type=1, G=2, P=4, N=8, K=16, offsets=FAKE, order=FAKE, per_row=2, rows=2, X=FAKE, ldx=16, dY=FAKE, lddy=8,
                dW=FAKE, lddw=8, stride_dw=128)
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_grouped_grad_w(**{**base, **change}) == want


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(k=-1), "DIM"), (dict(ldy=7), "LD"), (dict(ldo=7), "LD"), (dict(position=0), "NULL"),
    (dict(Y=0), "NULL"), (dict(out=0), "NULL"), (dict(weight=FAKE + 2), "ALIGN"), (dict(T=0, out=0), None)])
def test_combine_refuses(change, rc):
    base = dict(type=2, T=3, k=2, N=8, P=6, position=FAKE, weight=0, Y=FAKE, ldy=8, out=FAKE, ldo=8)
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_combine(**{**base, **change}) == want


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(T=-1), "DIM"), (dict(ldy=7), "LD"), (dict(lddo=7), "LD"), (dict(lddy=7), "LD"),
    (dict(position=0), "NULL"), (dict(dout=0), "NULL"), (dict(Y=0), "NULL"), (dict(dY=FAKE + 1), "ALIGN"),
    (dict(dY=0, dweight=0), None), (dict(k=0), None)])
def test_combine_grad_refuses(change, rc):
    base = dict(type=2, T=3, k=2, N=8, P=6, position=FAKE, weight=0, Y=FAKE, ldy=8, dout=FAKE, lddo=8, dY=FAKE, lddy=8,
                dweight=FAKE)
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_combine_grad(**{**base, **change}) == want


ADAPTERS = dict(type=1, T=4, N=8, K=16, R=8, n=2, X=FAKE, ldx=16, W=FAKE, ldw=8, A=FAKE, lda=8, stride_a=128, B=FAKE,
                ldb=8, stride_b=64, adapter=FAKE, scale=0, Y=FAKE, ldy=8, workspace=FAKE, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(T=-1), "DIM"), (dict(R=-1), "DIM"), (dict(R=257, lda=257), "DIM"), (dict(n=-1), "DIM"),
    (dict(ldx=15), "LD"), (dict(ldw=7), "LD"), (dict(lda=7), "LD"), (dict(ldb=7), "LD"), (dict(ldy=7), "LD"),
    (dict(stride_a=127), "LD"), (dict(stride_b=63), "LD"), (dict(X=0), "NULL"), (dict(B=0), "NULL"), (dict(A=0), "NULL"),
    (dict(adapter=0), "NULL"), (dict(Y=0), "NULL"), (dict(A=FAKE + 1), "ALIGN"), (dict(scale=FAKE + 2), "ALIGN"),
    (dict(workspace=0), "WORKSPACE"), (dict(workspace_bytes=0), "WORKSPACE"), (dict(workspace=FAKE + 8), "WORKSPACE"),
    (dict(T=0, Y=0, X=0), None), (dict(N=0, Y=0, W=0), None)])
def test_adapters_refuses(change, rc):
    want = gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)
    assert gb.gemm_f32_adapters(**{**ADAPTERS, **change}) == want


def test_adapters_workspace():
    assert gb.gemm_f32_adapters_ws_size(0, 8, 8, 8, -1) == gb.gemm_f32_adapters_ws_size(0, 0, 8, 8, 4) == 0
    assert gb.gemm_f32_adapters_ws_size(7, 8, 8, 8, 4) == 0
    for type_ in (0, 1, 2):
        assert gb.gemm_f32_adapters_ws_size(type_, 8, 8, 8, 4) % 16 == 0 < gb.gemm_f32_adapters_ws_size(type_, 8, 8, 8, 4)


def test_sizes_that_overflow_a_c_int_are_refused():
    with pytest.raises(ValueError, match="32-bit"):
        gb.gemm_f32_grouped(**{**GROUPED, "P": 1 << 32})
    with pytest.raises(ValueError, match="32-bit"):
        gb.gemm_f32_adapters(**{**ADAPTERS, "ldx": 1 << 33})


def test_torch_functions_refuse_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        gb.route(x, 2)
    with pytest.raises(TypeError):
        gb.route(x.double(), 2)
    with pytest.raises(ValueError):
        gb.route(x[0], 2)
    with pytest.raises(TypeError):
        gb.route_grad(x, i, torch.zeros(4, 2))
    with pytest.raises(TypeError):
        gb.expert_map(i, 4)
    with pytest.raises(TypeError):
        gb.grouped_matmul(x, torch.zeros(2, 8, 3), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gb.grouped_grad_x(x, torch.zeros(2, 3, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gb.grouped_grad_w(x, x, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gb.combine(x, i)
    with pytest.raises(TypeError):
        gb.combine_grad(x, x, i)
    with pytest.raises(TypeError):
        gb.adapter_matmul(x, torch.zeros(8, 3), torch.zeros(1, 8, 2), torch.zeros(1, 2, 3), torch.zeros(4, dtype=torch.int32))


# --- the oracle against itself ------------------------------------------------
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_oracle_route_gradient_against_differences(score, normalize):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(5, 9, generator=g, dtype=torch.float64)
    l[1, 4] = -oracle.INF
    weight, index, _ = oracle.route(l, 3, score=score, normalize=normalize, scale=1.5)
    assert torch.allclose(weight, oracle.route_weight_of(l, index, score, normalize, 1.5), rtol=1e-13, atol=0)
    dw = torch.randn(5, 3, generator=g, dtype=torch.float64)
    grad = oracle.route_grad(l, index, dw, score, normalize, 1.5)
    h = 1e-5
    for t in range(5):
        for e in range(9):
            if l[t, e] == -oracle.INF:
                continue
            up, down = l.clone(), l.clone()
            up[t, e] += h
            down[t, e] -= h
            d = sum(float((oracle.route_weight_of(x, index, score, normalize, 1.5) * dw).sum()) * s
                    for x, s in ((up, 1), (down, -1))) / (2 * h)
            # central differences: h^2 f''' / 6 and 2^-52 / h, both under 1e-9 here
            assert abs(d - float(grad[t, e])) < 1e-8


def test_oracle_expert_map():
    index = torch.tensor([[2, 0], [1, 2], [-1, 0], [7, 2]], dtype=torch.int32)
    offsets, order, position = oracle.expert_map(index, 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert order.tolist() == [1, 5, 2, 0, 3, 7, -1, -1]
    assert position.tolist() == [[3, 0], [2, 4], [-1, 1], [-1, 5]]


def test_oracle_route_ties_masks_and_groups():
    n = float("nan")
    l = torch.tensor([[1., 1., 1., 1.], [-oracle.INF, 0., -oracle.INF, 0.], [-oracle.INF] * 4, [0., n, 2., n]])
    w, i, _ = oracle.route(l, 3, normalize=True)
    assert i.tolist() == [[0, 1, 2], [1, 3, -1], [-1, -1, -1], [1, 3, 2]]
    assert w[1].tolist() == [0.5, 0.5, 0.0] and w[2].tolist() == [0, 0, 0] and w[3].isnan().all()
    l = torch.tensor([[5., 0., 3., 3.]])
    assert oracle.route(l, 2, groups=2, keep_groups=1, group_top=1)[1].tolist() == [[0, 1]]
    bias = torch.tensor([0., 0., 0.6, 0.6])
    assert oracle.route(l, 2, bias=bias, score="sigmoid", groups=2, keep_groups=1, group_top=2)[1].tolist() == [[2, 3]]


# --- sizes next to 2^31 -----------------------------------------------------------
MOST = 2 ** 31 - 4096


@pytest.mark.parametrize("size", [MOST + 1, 2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("fn,args", [
    ("grouped", dict(GROUPED, K="size", ldx="size", stride_w="size * 8", W=0)),
    ("grouped", dict(GROUPED, N="size", ldw="size", ldy="size", stride_w="size * 16", W=0)),
    ("grouped", dict(GROUPED, P="size", W=0)),
    ("grouped_grad_x", dict(type=1, G=2, P=4, N="size", K=16, offsets=FAKE, dY=FAKE, lddy="size", W=0, ldw="size", stride_w="size * 16",
                            dX=FAKE, lddx=16)),
    ("grouped_grad_w", dict(type=1, G=2, P="size", N=8, K=16, offsets=FAKE, order=FAKE, per_row=2, rows=2, X=FAKE, ldx=16, dY=0, lddy=8,
                            dW=FAKE, lddw=8, stride_dw=128)),
    ("combine", dict(type=2, T=3, k=2, N="size", P=6, position=FAKE, weight=0, Y=0, ldy="size", out=FAKE, ldo="size")),
    ("combine", dict(type=2, T=3, k="size", N=8, P=6, position=FAKE, weight=0, Y=0, ldy=8, out=FAKE, ldo=8)),
    ("combine_grad", dict(type=2, T=3, k=2, N="size", P=6, position=FAKE, weight=0, Y=0, ldy="size", dout=FAKE, lddo="size", dY=FAKE,
                          lddy="size", dweight=FAKE)),
    ("adapters", dict(ADAPTERS, K="size", ldx="size", stride_a="size * 8", W=0)),
    ("adapters", dict(ADAPTERS, N="size", ldw="size", ldb="size", ldy="size", stride_b="size * 8", W=0)),
])
def test_sizes_that_loops_would_step_past_2_31_are_refused(fn, args, size):
    """Kernels count along a size in 32 bits and step past it: 2^31 - 4096 is the largest.  (A NULL operand
    keeps a call that is not refused for its size from being launched.)"""
    change = {k: eval(v, {"size": size}) if isinstance(v, str) else v for k, v in args.items()}
    assert getattr(gb, "gemm_f32_" + fn)(**change) == gb.GEMM_F32_ERR_DIM


@pytest.mark.parametrize("fn,args", [
    ("grouped", dict(GROUPED, K=MOST, ldx=MOST, stride_w=MOST * 8, W=0)),
    ("combine", dict(type=2, T=3, k=2, N=MOST, P=6, position=FAKE, weight=0, Y=0, ldy=MOST, out=FAKE, ldo=MOST)),
    ("adapters", dict(ADAPTERS, K=MOST, ldx=MOST, stride_a=MOST * 8, W=0))])
def test_the_largest_sizes_are_taken(fn, args):
    assert getattr(gb, "gemm_f32_" + fn)(**args) == gb.GEMM_F32_ERR_NULL


# --- streams and integers that the torch functions are given ------------------------
def test_a_stream_of_another_device_is_refused():
    """Run on the tensors' device, the call would ignore the stream; on the stream's, the tensors'."""
    class Stream:
        device = torch.device("cuda", 1)
    ran = []
    with pytest.raises(ValueError, match="stream"):
        gb._call_on(torch.device("cuda", 0), Stream(), lambda: ran.append(1))
    assert not ran


@pytest.mark.parametrize("value", [-(1 << 32) + 1, -(1 << 31) - 1, 1 << 31, (1 << 32) + 1])
def test_integers_that_would_wrap_to_valid_ones_are_refused(value):
    """ctypes passes the low 32 bits: -(2^32) + 1 groups would be one."""
    with pytest.raises(ValueError, match="32-bit"):
        gb._fit(4, 8, value)


def test_first_calls_of_two_threads(monkeypatch):
    """A thread that finds the other one half way through _here()'s first call looks the functions up itself."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 77 + index, raising=False)
    monkeypatch.setattr(gb, "_current_device", lambda: 0)      # set by the other thread, which has not come further
    monkeypatch.setattr(gb, "_current_raw_stream", None)
    assert gb._here(torch.device("cuda", 3)) == 80


@pytest.mark.parametrize("fn,args", [
    ("grouped", dict(GROUPED, P=1 << 30, N=1 << 20, X=0)),                    # and NULL, and short rows
    ("grouped_grad_x", dict(type=0, G=2, P=1 << 30, N=8, K=1 << 20, offsets=FAKE, dY=0, lddy=1, W=FAKE, ldw=1, stride_w=1, dX=FAKE, lddx=16)),
    ("grouped_grad_w", dict(type=1, G=1 << 20, P=4, N=1 << 12, K=1 << 12, offsets=0, order=0, per_row=2, rows=4, X=FAKE, ldx=1, dY=FAKE,
                            lddy=8, dW=FAKE, lddw=8, stride_dw=128)),
    # more tiles than 64 bits count
    ("grouped_grad_w", dict(type=0, G=(1 << 31) - 1, P=4, N=1 << 30, K=1 << 30, offsets=0, order=0, per_row=2, rows=4, X=FAKE, ldx=1 << 30,
                            dY=FAKE, lddy=1 << 30, dW=FAKE, lddw=1 << 30, stride_dw=1 << 60)),
    ("adapters", dict(ADAPTERS, T=1 << 25, N=1 << 30, Y=0)),
])
def test_too_many_tiles_are_refused_with_the_sizes(fn, args):
    """Sizes come before leading dimensions and pointers, whatever else is wrong."""
    assert getattr(gb, "gemm_f32_" + fn)(**args) == gb.GEMM_F32_ERR_DIM


def test_the_poisoned_build_covers_every_panel_load():
    """Every direct load into LDS stands behind poison_slots() in its function."""
    src = open(os.path.join(ROOT, "dense_fp32_gemm_amd", "csrc", "rows_tile.h")).read()
    assert "#ifdef GEMM_F32_POISON_LDS" in src
    fires = re.split(r"__device__ inline void fire\(", src)[1:]
    assert len(fires) == 2 == src.count("__builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc")
    for body in fires:
        body = body[:body.index("\n    }\n")]
        assert "poison_slots<" in body and "buffer_load_lds(" in body
    for name in ("rows_adapters.hip", "rows_grouped.hip", "rows_route.hip", "rows_common.h"):
        assert "buffer_load_lds" not in open(os.path.join(ROOT, "dense_fp32_gemm_amd", "csrc", name)).read()
