"""CPU checks of the operators of a feed-forward block: refusals, workspace
sizes, the declared ABI, and the oracle's own gradients against differences."""
import os
import re
import subprocess

import pytest

from dense_fp32_gemm_amd import binding as gb
import ffn_oracle as oracle

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f32_ffn.h")
FAKE = 0x100000
MOST = 2 ** 31 - 4096


def code(rc):
    return gb.GEMM_F32_OK if rc is None else getattr(gb, "GEMM_F32_ERR_" + rc)


def test_library_exports_and_binds_every_declared_function():
    names = sorted(set(re.findall(r"GEMM_F32_API\s+[\w\s\*]*?\b(gemm_f32\w*)\s*\(", open(HEADER).read())))
    assert len(names) == 8, names
    for n in names:
        assert hasattr(gb.load(), n) and hasattr(gb, n), n


def test_constants_match_the_header():
    found = re.findall(r"#define (GEMM_F32_(?:GATE|MAX)_\w+)\s+(\d+)", open(HEADER).read())
    assert len(found) == 5
    for name, value in found:
        assert getattr(gb, name) == int(value), name


NORM = dict(type=1, T=4, N=8, X=FAKE, ldx=8, residual=FAKE, ldr=8, weight=FAKE, eps=1e-6, sum=FAKE, lds=8)
BAD_NORM = [
    (dict(type=3), "TYPE"), (dict(type=-1), "TYPE"), (dict(T=-1), "DIM"), (dict(N=-1), "DIM"), (dict(T=MOST + 1), "DIM"),
    (dict(N=MOST + 1, ldx=MOST + 1), "DIM"), (dict(ldx=7), "LD"), (dict(ldr=7), "LD"), (dict(lds=7), "LD"), (dict(eps=0.0), "OPTION"),
    (dict(eps=-1e-6), "OPTION"), (dict(eps=float("nan")), "OPTION"), (dict(eps=float("inf")), "OPTION"), (dict(X=0), "NULL"),
    (dict(X=FAKE + 1), "ALIGN"), (dict(residual=FAKE + 1), "ALIGN"), (dict(sum=FAKE + 1), "ALIGN"), (dict(weight=FAKE + 2), "ALIGN"),
    (dict(T=0, X=0), None)]


@pytest.mark.parametrize("change,rc", BAD_NORM + [
    (dict(ldy=7), "LD"), (dict(Y=0), "NULL"), (dict(Y=FAKE + 1), "ALIGN"), (dict(N=0, X=0, Y=0), None),
    (dict(type=7, T=-1, ldx=0), "TYPE"), (dict(ldy=7, eps=0.0, X=0), "LD")])
def test_rms_norm_refuses(change, rc):
    assert gb.gemm_f32_rms_norm(**{**NORM, "Y": FAKE, "ldy": 8, **change}) == code(rc)


@pytest.mark.parametrize("change,rc", BAD_NORM + [
    (dict(ldq=7), "LD"), (dict(Q=0), "NULL"), (dict(scale=0), "NULL"), (dict(scale=FAKE + 2), "ALIGN")])
def test_rms_norm_int8_refuses(change, rc):
    assert gb.gemm_f32_rms_norm_int8(**{**NORM, "Q": FAKE, "ldq": 8, "scale": FAKE, **change}) == code(rc)


@pytest.mark.parametrize("change,rc", [
    (dict(type=3), "TYPE"), (dict(T=-1), "DIM"), (dict(N=MOST + 1), "DIM"), (dict(lddy=7), "LD"), (dict(lds=7), "LD"), (dict(ldds=7), "LD"),
    (dict(lddx=7), "LD"), (dict(eps=0.0), "OPTION"), (dict(dY=0), "NULL"), (dict(S=0), "NULL"), (dict(dY=FAKE + 1), "ALIGN"),
    (dict(dsum=FAKE + 1), "ALIGN"), (dict(dX=FAKE + 1), "ALIGN"), (dict(dweight=FAKE + 2), "ALIGN"), (dict(weight=FAKE + 1), "ALIGN"),
    (dict(workspace=0), "WORKSPACE"), (dict(workspace=FAKE + 8), "WORKSPACE"), (dict(workspace_bytes=16), "WORKSPACE"),
    (dict(dX=0, dweight=0), None), (dict(N=0, dY=0), None), (dict(T=0, dweight=0), None)])
def test_rms_norm_grad_refuses(change, rc):
    base = dict(type=1, T=4, N=8, dY=FAKE, lddy=8, S=FAKE, lds=8, weight=FAKE, eps=1e-6, dsum=FAKE, ldds=8, dX=FAKE, lddx=8, dweight=FAKE,
                workspace=FAKE, workspace_bytes=1 << 20)
    assert gb.gemm_f32_rms_norm_grad(**{**base, **change}) == code(rc)


def test_rms_norm_grad_workspace():
    assert gb.gemm_f32_rms_norm_grad_ws_size(0, 8) == gb.gemm_f32_rms_norm_grad_ws_size(8, 0) == gb.gemm_f32_rms_norm_grad_ws_size(-1, 8) == 0
    for T, N in [(1, 1), (5, 7), (4000, 100)]:
        assert gb.gemm_f32_rms_norm_grad_ws_size(T, N) % 16 == 0 < gb.gemm_f32_rms_norm_grad_ws_size(T, N)
    # bounded by the number of workgroups, not by the rows
    assert gb.gemm_f32_rms_norm_grad_ws_size(1 << 20, 4096) == gb.gemm_f32_rms_norm_grad_ws_size(1 << 30, 4096) <= 4096 * 4096 * 4


@pytest.mark.parametrize("change,rc", [
    (dict(type=3), "TYPE"), (dict(T=-1), "DIM"), (dict(N=MOST + 1), "DIM"), (dict(gate=1, N=MOST // 2 + 1), "DIM"), (dict(ldx=7), "LD"),
    (dict(gate=1, ldx=15), "LD"), (dict(ldq=7), "LD"), (dict(gate=4), "OPTION"), (dict(gate=-1), "OPTION"), (dict(X=0), "NULL"),
    (dict(Q=0), "NULL"), (dict(scale=0), "NULL"), (dict(X=FAKE + 1), "ALIGN"), (dict(scale=FAKE + 2), "ALIGN"), (dict(T=0, X=0, Q=0, scale=0), None)])
def test_quantize_refuses(change, rc):
    base = dict(type=1, gate=0, T=4, N=8, X=FAKE, ldx=16, Q=FAKE, ldq=8, scale=FAKE)
    assert gb.gemm_f32_quantize(**{**base, **change}) == code(rc)


INT8 = dict(type=1, T=4, N=8, K=16, Q=FAKE, ldq=16, scale=FAKE, W=FAKE, ldw=16, w_scale=FAKE, bias=FAKE, Y=FAKE, ldy=8)


@pytest.mark.parametrize("change,rc", [
    (dict(type=3), "TYPE"), (dict(T=-1), "DIM"), (dict(N=-1), "DIM"), (dict(K=-1), "DIM"), (dict(K=131072, ldq=131072, ldw=131072), "DIM"),
    (dict(T=MOST + 1), "DIM"), (dict(T=1 << 30, N=1 << 20, ldy=1), "DIM"), (dict(ldq=15), "LD"), (dict(ldw=15), "LD"), (dict(ldy=7), "LD"),
    (dict(Q=0), "NULL"), (dict(W=0), "NULL"), (dict(scale=0), "NULL"), (dict(w_scale=0), "NULL"), (dict(Y=0), "NULL"),
    (dict(scale=FAKE + 1), "ALIGN"), (dict(w_scale=FAKE + 2), "ALIGN"), (dict(bias=FAKE + 2), "ALIGN"), (dict(Y=FAKE + 1), "ALIGN"),
    (dict(T=0, Q=0, Y=0), None), (dict(N=0, W=0, Y=0), None)])
def test_int8_refuses(change, rc):
    assert gb.gemm_f32_int8(**{**INT8, **change}) == code(rc)


def test_int8_sums_fit_at_the_largest_depth():
    assert 128 * 128 * gb.GEMM_F32_MAX_INT8_DEPTH < 2 ** 31 <= 128 * 128 * (gb.GEMM_F32_MAX_INT8_DEPTH + 1)


GATED = dict(type=1, gate=1, G=2, P=4, N=8, K=16, offsets=FAKE, order=FAKE, per_row=2, rows=2, X=FAKE, ldx=16, W=FAKE, ldw=16,
             stride_w=256, H=FAKE, ldh=8, pre=FAKE, ldp=16)


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(G=-1), "DIM"), (dict(P=-1), "DIM"), (dict(N=-1), "DIM"), (dict(K=-1), "DIM"), (dict(rows=-1), "DIM"),
    (dict(order=0), "DIM"), (dict(N=MOST // 2 + 1), "DIM"), (dict(K=MOST + 1), "DIM"), (dict(P=1 << 30, N=1 << 20), "DIM"), (dict(ldx=15), "LD"),
    (dict(ldw=15), "LD"), (dict(ldh=7), "LD"), (dict(ldp=15), "LD"), (dict(stride_w=255), "LD"), (dict(gate=0), "OPTION"), (dict(gate=4), "OPTION"),
    (dict(per_row=0), "OPTION"), (dict(offsets=0), "NULL"), (dict(X=0), "NULL"), (dict(W=0), "NULL"), (dict(H=0), "NULL"),
    (dict(X=FAKE + 1), "ALIGN"), (dict(order=FAKE + 2), "ALIGN"), (dict(pre=FAKE + 1), "ALIGN"),
    (dict(G=0, offsets=0, H=0), None), (dict(P=0, H=0), None), (dict(N=0, H=0, W=0), None)])
def test_gated_refuses(change, rc):
    assert gb.gemm_f32_gated(**{**GATED, **change}) == code(rc)


@pytest.mark.parametrize("change,rc", [
    (dict(type=9), "TYPE"), (dict(P=-1), "DIM"), (dict(N=-1), "DIM"), (dict(N=MOST // 2 + 1), "DIM"), (dict(ldp=15), "LD"), (dict(lddh=7), "LD"),
    (dict(lddp=15), "LD"), (dict(gate=0), "OPTION"), (dict(gate=9), "OPTION"), (dict(pre=0), "NULL"), (dict(dH=0), "NULL"), (dict(dpre=0), "NULL"),
    (dict(pre=FAKE + 1), "ALIGN"), (dict(dH=FAKE + 1), "ALIGN"), (dict(dpre=FAKE + 1), "ALIGN"), (dict(P=0, pre=0), None), (dict(N=0, dH=0), None)])
def test_gate_grad_refuses(change, rc):
    base = dict(type=1, gate=1, P=4, N=8, pre=FAKE, ldp=16, dH=FAKE, lddh=8, dpre=FAKE, lddp=16)
    assert gb.gemm_f32_gate_grad(**{**base, **change}) == code(rc)


@pytest.mark.parametrize("fn,args", [
    ("grouped", dict(type=1, G=0, P=4, N=8, K=16, offsets=0, order=0, per_row=1, rows=4, X=FAKE, ldx=16, W=FAKE, ldw=8, stride_w=128, Y=FAKE, ldy=8)),
    ("grouped_grad_x", dict(type=1, G=3, P=4, N=8, K=16, offsets=0, dY=FAKE, lddy=8, W=FAKE, ldw=8, stride_w=128, dX=FAKE, lddx=16)),
    ("grouped_grad_w", dict(type=1, G=2, P=4, N=8, K=16, offsets=0, order=0, per_row=1, rows=4, X=FAKE, ldx=16, dY=FAKE, lddy=8, dW=FAKE, lddw=8,
                            stride_dw=128)),
    # one group of all places: the next check is reached
    ("grouped", dict(type=1, G=1, P=4, N=8, K=16, offsets=0, order=0, per_row=1, rows=4, X=FAKE + 1, ldx=16, W=FAKE, ldw=8, stride_w=0, Y=FAKE, ldy=8)),
    ("grouped_grad_x", dict(type=1, G=1, P=4, N=8, K=16, offsets=0, dY=FAKE + 1, lddy=8, W=FAKE, ldw=8, stride_w=0, dX=FAKE, lddx=16)),
    ("grouped_grad_w", dict(type=1, G=1, P=4, N=8, K=16, offsets=0, order=0, per_row=1, rows=4, X=FAKE + 1, ldx=16, dY=FAKE, lddy=8, dW=FAKE,
                            lddw=8, stride_dw=0))])
def test_offsets_may_be_left_out_with_one_group_only(fn, args):
    want = None if args["G"] == 0 else "ALIGN" if args["G"] == 1 else "NULL"
    assert getattr(gb, "gemm_f32_" + fn)(**args) == code(want)


def test_sizes_that_overflow_a_c_int_are_refused():
    with pytest.raises(ValueError, match="32-bit"):
        gb.gemm_f32_int8(**{**INT8, "K": 1 << 32})
    with pytest.raises(ValueError, match="32-bit"):
        gb.gemm_f32_gated(**{**GATED, "ldp": 1 << 33})
    with pytest.raises(ValueError, match="32-bit"):
        gb.gemm_f32_rms_norm(**{**NORM, "Y": FAKE, "ldy": 1 << 32})


def test_torch_functions_refuse_cpu_tensors_and_wrong_arguments():
    x, q = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8)
    with pytest.raises(TypeError):
        gb.rms_norm(x)
    with pytest.raises(TypeError):
        gb.rms_norm_int8(x)
    with pytest.raises(TypeError):
        gb.rms_norm(x.double())
    with pytest.raises(ValueError):
        gb.rms_norm(x[0])
    with pytest.raises(TypeError):
        gb.rms_norm_grad(x, x)
    with pytest.raises(TypeError):
        gb.quantize(x)
    with pytest.raises(TypeError):
        gb.int8_matmul(q, torch.zeros(4), q, torch.zeros(4))
    with pytest.raises(TypeError):
        gb.gated_matmul(x, torch.zeros(1, 8, 6))
    with pytest.raises(TypeError):
        gb.gate_grad(x[:, :4], x)
    with pytest.raises(ValueError, match="gate"):
        gb._gate("tanh")
    with pytest.raises(ValueError, match="gate"):
        gb._gate([])


def test_the_direct_loads_stand_in_one_file():
    """So that the poisoned build covers them (test_rows_cpu.py)."""
    folder = os.path.join(ROOT, "dense_fp32_gemm_amd", "csrc")
    for name in os.listdir(folder):
        if name.startswith("ffn_"):
            assert "load_lds" not in open(os.path.join(folder, name)).read(), name


EACH_CHUNK = r"""
#include <stdio.h>
#include <stdlib.h>
#include "ffn_rows.h"

// Whether a thread's columns are those of its chunks, one after the other, and end with the row.
template <int TPR, class E>
static void walk(int N)
{
    const int step = TPR * E::kChunk, js[] = {0, 1, TPR / 2 - 1, TPR / 2, TPR - 1};
    for (int j : js) {
        int64_t next = j * E::kChunk;
        ffn::each_chunk<TPR, 0, E>(N, j, [&](int, int n0) {
            if (n0 != next || n0 >= N) {
                printf("%d threads of %d elements, N = %d, thread %d: column %d after %lld\n", TPR, (int)E::kChunk, N, j, n0,
                       (long long)(next - step));
                exit(1);
            }
            next += step;
        });
        if (next < N)
            exit(2);
    }
}

int main()
{
    const int most = rows::kMaxSize;
    for (int N : {0, 1, 20000, most - 8192, most - 4096, most - 4095, most - 1, most}) {
        walk<1024, rows::F32>(N);
        walk<1024, rows::Bf16>(N);
        walk<1024, rows::F16>(N);
    }
    return 0;
}
"""


def test_rows_of_the_largest_sizes_end(tmp_path):
    """The loop over a row that does not fit the registers, on the host, up to the largest size that is taken
    (-fwrapv: an index that passes 2^31 comes out negative, as on the GPU)."""
    src, exe = tmp_path / "each_chunk.hip", tmp_path / "each_chunk"
    src.write_text(EACH_CHUNK)
    csrc = os.path.join(ROOT, "dense_fp32_gemm_amd", "csrc")
    subprocess.run(["hipcc", "-O1", "-fwrapv", "-std=c++17", "--offload-host-only", "-I", csrc, "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True, capture_output=True, timeout=300)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


# --- the oracle against itself --------------------------------------------------------
def difference(f, x, h=1e-5):
    """The derivative of f (a number) by each element of x, by differences."""
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        up, down = x.clone(), x.clone()
        up.view(-1)[i] += h
        down.view(-1)[i] -= h
        out.view(-1)[i] = (f(up) - f(down)) / (2 * h)
    return out


def test_oracle_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    S, d, w = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 7), (3, 7), (7,)))
    S[1] = 0
    dX, dw = oracle.norm_grad(d.float(), S.float(), w.float(), 0.1, None)[:2]
    S, d, w = S.float().double(), d.float().double(), w.float().double()
    # h^2 f''' / 6 and 2^-52 / h: both under 1e-9
    assert (difference(lambda s: (oracle.normed(s, w, 0.1) * d).sum(), S) - dX).abs().max() < 1e-7
    assert (difference(lambda v: (oracle.normed(S, v, 0.1) * d).sum(), w) - dw).abs().max() < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_oracle_gate_gradient_against_differences(kind):
    g = torch.Generator().manual_seed(2)
    pre, d = torch.randn(3, 8, generator=g) * 3, torch.randn(3, 4, generator=g)
    want = oracle.gate_grad(d, pre, kind)[0]
    got = difference(lambda p: (oracle.gate(p[:, :4], kind) * p[:, 4:] * d.double()).sum(), pre.double())
    assert (got - want).abs().max() < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_oracle_gates_against_torch(kind):
    x = torch.linspace(-9, 9, 181, dtype=torch.float64)
    want = {"silu": torch.nn.functional.silu(x), "gelu": torch.nn.functional.gelu(x),
            "gelu_tanh": torch.nn.functional.gelu(x, approximate="tanh")}[kind]
    # torch's forms lose a few 2^-53 of |x| to cancellation on the left
    assert (oracle.gate(x, kind) - want).abs().max() < 1e-14


def test_oracle_rows_in_8_bits():
    y = torch.tensor([[127.0, 0.5, 1.5, -2.5, 0.0], [0.0] * 5, [1.0, oracle.INF, 0, 0, 0], [1.0, float("nan"), 0, 0, 0], [1e-44, 0, 0, 0, 0]],
                     dtype=torch.float64)
    Q, s = oracle.int8_rows(y)
    assert Q.tolist() == [[127, 0, 2, -2, 0], [0] * 5, [0] * 5, [0] * 5, [0] * 5]
    assert s[0] == 1 and s[1] == s[4] == 2.0 ** -126 and s[2].isnan() and s[3].isnan()
