"""The operators' argument checks (CPU only): the C ABI with addresses that are never
dereferenced, and the Python binding with CPU tensors.  Nothing here reaches a launch."""
import ctypes
import os
import re

import pytest
import torch

import sparse_mixture_experts_ffn_b200 as moe
from sparse_mixture_experts_ffn_b200 import build, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


def shape(R=64, N=128, K=256, E=4, dtype=moe.MOE_BF16):
    return ops.MoEGemmShape(R, N, K, E, dtype)


def test_the_shape_structure_matches_the_header():
    text = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
    body = re.search(r"typedef struct \{(.*?)\}\s*moe_gemm_shape;", text, flags=re.S).group(1)
    fields = []
    for decl in body.split(";"):
        if decl.strip():
            ctype, names = decl.strip().split(None, 1)
            fields += [(n.strip(), ctype) for n in names.split(",")]
    sizes = {"int64_t": 8, "int32_t": 4}
    assert [(f, ctypes.sizeof(t)) for f, t in ops.MoEGemmShape._fields_] == [(f, sizes[c]) for f, c in fields]


BAD_SHAPES = [(dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(E=0), INVALID),
              (dict(dtype=2), INVALID), (dict(N=132), UNSUPPORTED), (dict(K=100), UNSUPPORTED),
              (dict(E=1025), UNSUPPORTED), (dict(R=2 ** 30 + 1), UNSUPPORTED), (dict(N=2 ** 20 + 8), UNSUPPORTED)]


@pytest.mark.parametrize("entry", ["moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad"])
def test_grouped_products_reject_bad_arguments(lib, entry):
    fn = getattr(lib, entry)
    for kw, want in BAD_SHAPES:
        assert fn(shape(**kw), 16, 32, 16, 48, None) == want, kw
    assert fn(None, 16, 32, 16, 48, None) == INVALID
    for ptrs in ((None, 32, 16, 48), (16, None, 16, 48), (16, 32, None, 48), (16, 32, 16, None), (24, 32, 16, 48),
                 (16, 24, 16, 48), (16, 32, 18, 48), (16, 32, 16, 8), (16, 32, 16, 16), (16, 32, 16, 32)):
        assert fn(shape(), *ptrs, None) == INVALID, ptrs
    if entry != "moe_grouped_gemm_wgrad":  # no rows: nothing to do, nothing looked at
        assert fn(shape(R=0), None, None, None, None, None) == OK
    else:
        assert fn(shape(R=0), None, None, None, 16, None) == INVALID


def test_linear_rejects_bad_arguments(lib):
    def call(s=None, x=16, W=32, bias=None, res=None, act=0, y=48, z=None):
        return lib.moe_linear(s or shape(E=1), x, W, bias, res, act, y, z, None)
    for kw, want in BAD_SHAPES:
        kw = {"E": 1, **kw}
        assert call(shape(**kw)) == want, kw
    assert call(shape(E=2)) == INVALID
    for kw in (dict(x=None), dict(W=None), dict(y=None), dict(x=8), dict(W=24), dict(y=40), dict(bias=2), dict(res=8),
               dict(z=8), dict(z=48), dict(z=16), dict(res=64, z=64), dict(y=16), dict(y=32), dict(act=-1), dict(act=5)):
        assert call(**kw) == INVALID, kw
    assert call(shape(E=1, R=0), x=None) == OK


def test_linear_backward_rejects_bad_arguments(lib):
    s = shape(E=1)
    need = lib.moe_linear_backward_workspace_bytes(s, 2, 1)
    assert need >= 64 * 128 * 2 and need % 256 == 0
    assert lib.moe_linear_backward_workspace_bytes(s, 0, 0) == 0
    assert lib.moe_linear_backward_workspace_bytes(shape(E=2), 2, 1) == 0
    assert lib.moe_linear_backward_workspace_bytes(s, 9, 1) == 0

    def call(s=s, dy=16, x=16, W=16, z=16, act=2, dx=16, dW=16, db=4, ws=256, nb=need):
        return lib.moe_linear_backward(s, dy, x, W, z, act, dx, dW, db, ws, nb, None)
    for kw in (dict(dy=None), dict(x=None), dict(W=None), dict(z=None), dict(ws=None), dict(ws=128), dict(dx=8),
               dict(dW=24), dict(db=2), dict(act=7), dict(s=shape(E=3)), dict(dy=24), dict(z=8)):
        assert call(**kw) == INVALID, kw
    assert call(nb=need - 1) == TOO_SMALL
    assert call(s=shape(E=1, N=100)) == UNSUPPORTED
    # nothing asked for: nothing to do, and no workspace for the bias gradient
    assert call(dx=None, dW=None, db=None) == OK


def test_swiglu_rejects_bad_arguments(lib):
    nan, inf = float("nan"), float("inf")
    for R, I, dt, limit, want in ((-1, 8, 1, 0, INVALID), (4, 0, 1, 0, INVALID), (4, 8, 7, 0, INVALID),
                                  (4, 8, 1, -1.0, INVALID), (4, 8, 1, nan, INVALID), (4, 8, 1, inf, INVALID),
                                  (4, 12, 1, 0, UNSUPPORTED), (2 ** 30 + 1, 8, 1, 0, UNSUPPORTED),
                                  (4, 2 ** 20 + 8, 1, 0, UNSUPPORTED), (0, 8, 1, 0, OK)):
        assert lib.moe_swiglu(R, I, dt, 16, None, limit, 16, None) == want
        assert lib.moe_swiglu_backward(R, I, dt, 16, 16, None, limit, 16, None, None) == want
    for gu, w, h in ((None, None, 16), (16, None, None), (8, None, 16), (16, 2, 16), (16, None, 24)):
        assert lib.moe_swiglu(4, 8, 1, gu, w, 0.0, h, None) == INVALID
        assert lib.moe_swiglu_backward(4, 8, 1, 16, gu, w, 0.0, h, None, None) == INVALID
    assert lib.moe_swiglu_backward(4, 8, 1, None, 16, None, 0.0, 16, None, None) == INVALID
    assert lib.moe_swiglu_backward(4, 8, 1, 16, 16, 4, 0.0, 16, 2, None) == INVALID


def test_overlapping_operands_are_refused(lib):
    """Outputs that touch an input or another output in part: R 64, N 128, K 256 in bf16 (x and dx
    32 KB, y and dy 16 KB, a weight 64 KB).  Only refused calls: the addresses are never used."""
    M = 1 << 20
    s, g = shape(E=1), shape(E=4)
    a, b, o = 4 * M, 8 * M, 12 * M  # far apart
    off = 16 * M
    rk, rn, w = 64 * 256 * 2, 64 * 128 * 2, 128 * 256 * 2
    for entry, n_rows, n_other, n_out in (("moe_grouped_gemm", rk, 4 * w, rn), ("moe_grouped_gemm_dgrad", rn, 4 * w, rk),
                                          ("moe_grouped_gemm_wgrad", rn, rk, 4 * w)):
        fn = getattr(lib, entry)
        for out in (a + n_rows - 16, a - n_out + 16, b + n_other - 16, b - n_out + 16, off, off - n_out + 16):
            assert fn(g, a, b, off, out, None) == INVALID, (entry, out)
    for kw in (dict(y=a + rk - 16), dict(y=b - rn + 16), dict(res=o + 16), dict(z=o - rn + 16), dict(z=o + rn - 16),
               dict(res=off, z=off + 16), dict(bias=o + rn - 4), dict(z=b + w - 16)):
        kw = {"res": None, "z": None, "bias": None, "y": o, **kw}
        assert lib.moe_linear(s, a, b, kw["bias"], kw["res"], 1, kw["y"], kw["z"], None) == INVALID, kw
    need = lib.moe_linear_backward_workspace_bytes(s, 2, 1)

    def back(dy=a, x=b, W=o, z=off, dx=20 * M, dW=24 * M, db=28 * M, ws=32 * M):
        return lib.moe_linear_backward(s, dy, x, W, z, 2, dx, dW, db, ws, need, None)
    for kw in (dict(dx=a), dict(dx=b), dict(dx=o + 16), dict(dx=off + rn - 16), dict(dW=a - 16), dict(dW=b), dict(dW=o),
               dict(dW=20 * M + 16), dict(db=20 * M), dict(db=24 * M + 4), dict(db=a), dict(ws=a), dict(ws=20 * M),
               dict(ws=28 * M), dict(ws=off), dict(dx=32 * M + 16)):
        assert back(**kw) == INVALID, kw
    ri = 4 * 8 * 2  # a row block of h: R 4, I 8
    for h in (a, a + 2 * ri - 16, a - ri + 16):
        assert lib.moe_swiglu(4, 8, 1, a, None, 0.0, h, None) == INVALID
    assert lib.moe_swiglu(4, 8, 1, a, o, 0.0, o, None) == INVALID
    for dgu, dw in ((a, None), (b, None), (a + ri - 16, None), (b + 16, None), (o, o + 4), (o, off), (o, a)):
        assert lib.moe_swiglu_backward(4, 8, 1, a, b, off, 0.0, dgu, dw, None) == INVALID


# ------------------------------------------------------------------ the binding
BF = torch.bfloat16
R, N, K, E = 6, 16, 24, 3


def bf(*s):
    return torch.zeros(*s, dtype=BF)


def offs(n=E + 1, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def test_consistent_tensors_fail_only_for_want_of_a_gpu():
    calls = [lambda: moe.grouped_gemm(bf(R, K), bf(E, N, K), offs()),
             lambda: moe.grouped_gemm_dgrad(bf(R, N), bf(E, N, K), offs()),
             lambda: moe.grouped_gemm_wgrad(bf(R, N), bf(R, K), offs()),
             lambda: moe.linear(bf(R, K), bf(N, K), bias=torch.zeros(N), residual=bf(R, N), activation="gelu"),
             lambda: moe.linear_backward(bf(R, N), bf(R, K), bf(N, K), preact=bf(R, N), activation="silu"),
             lambda: moe.swiglu(bf(R, 2 * N), row_w=torch.zeros(R), limit=7.0),
             lambda: moe.swiglu_backward(bf(R, N), bf(R, 2 * N))]
    for c in calls:
        with pytest.raises(ValueError, match="CUDA"):
            c()


@pytest.mark.parametrize("call, match", [
    (lambda: moe.grouped_gemm(bf(R, K + 8), bf(E, N, K), offs()), "row operand"),
    (lambda: moe.grouped_gemm(bf(R, K), torch.zeros(E, N, K), offs()), "W must be"),
    (lambda: moe.grouped_gemm(bf(R, K), bf(N, K), offs()), "2-D"),
    (lambda: moe.grouped_gemm(bf(R, K), bf(E, N, K), offs(E)), "offsets"),
    (lambda: moe.grouped_gemm(bf(R, K), bf(E, N, K), offs(dtype=torch.int64)), "offsets"),
    (lambda: moe.grouped_gemm(bf(R, K), bf(E, N, K), offs(), y=bf(R, K)), "y must be"),
    (lambda: moe.grouped_gemm(bf(R, K), bf(E, K, N).transpose(1, 2), offs()), "contiguous"),
    (lambda: moe.grouped_gemm(bf(K, R).t(), bf(E, N, K), offs()), "contiguous"),
    (lambda: moe.grouped_gemm(torch.zeros(R, K, dtype=torch.float16), bf(E, N, K), offs()), "bf16 or fp32"),
    (lambda: moe.grouped_gemm(bf(R, K), torch.zeros(E, N, K, dtype=BF, device="meta"), offs()), "meta"),
    (lambda: moe.grouped_gemm_dgrad(bf(R, K), bf(E, N, K), offs()), "row operand"),
    (lambda: moe.grouped_gemm_dgrad(bf(R, N), bf(E, N, K), offs(), dx=bf(R, N)), "dx must be"),
    (lambda: moe.grouped_gemm_wgrad(bf(R, N), bf(R + 1, K), offs()), "x must be"),
    (lambda: moe.grouped_gemm_wgrad(bf(R, N), bf(R, K), offs(1)), "offsets"),
    (lambda: moe.grouped_gemm_wgrad(bf(R, N), bf(R, K), offs(), dW=bf(E, K, N)), "dW must be"),
    (lambda: moe.linear(bf(R, K), bf(N, K + 8)), "W must be"),
    (lambda: moe.linear(bf(R, K), bf(N, K), bias=bf(N)), "bias must be"),
    (lambda: moe.linear(bf(R, K), bf(N, K), residual=bf(R, K)), "residual must be"),
    (lambda: moe.linear(bf(R, K), bf(N, K), activation="tanh"), "activation"),
    (lambda: moe.linear(bf(R, K), bf(N, K), preact=torch.zeros(R, N)), "preact must be"),
    (lambda: moe.linear_backward(bf(R, N), bf(R, K), bf(N, K), activation="relu"), "needs preact"),
    (lambda: moe.linear_backward(bf(R, N), bf(R, K), bf(N, K), input_grad=False, dx=bf(R, K)), "not asked"),
    (lambda: moe.linear_backward(bf(R, N), bf(R, K), bf(N, K), bias_grad=True, dbias=bf(N)), "dbias must be"),
    (lambda: moe.linear_backward(bf(R, K), bf(R, K), bf(N, K)), "x must be|W must be"),
    (lambda: moe.swiglu(bf(R, 2 * N + 1)), "gate_up must be"),
    (lambda: moe.swiglu(bf(R, 2 * N), row_w=bf(R)), "row_w must be"),
    (lambda: moe.swiglu(bf(R, 2 * N), limit=-1.0), "limit"),
    (lambda: moe.swiglu(bf(R, 2 * N), limit=float("nan")), "limit"),
    (lambda: moe.swiglu(bf(R, 2 * N), h=bf(R, 2 * N)), "h must be"),
    (lambda: moe.swiglu_backward(bf(R, 2 * N), bf(R, 2 * N)), "dh must be"),
    (lambda: moe.swiglu_backward(bf(R, N), bf(R, 2 * N), d_row_w=torch.zeros(R)), "without row_w"),
])
def test_mismatched_tensors_are_rejected(call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_sizes_that_would_wrap_in_32_bits_are_refused():
    """2^32 + 8 features would arrive as 8."""
    def big(*s, dtype=BF):
        return torch.empty(*s, dtype=dtype, device="meta")
    n, o = 2 ** 32 + 8, torch.empty(2, dtype=torch.int32, device="meta")
    for call in (lambda: moe.grouped_gemm(big(1, n), big(1, 8, n), o),
                 lambda: moe.grouped_gemm_dgrad(big(1, 8), big(1, 8, n), o),
                 lambda: moe.grouped_gemm_wgrad(big(1, n), big(1, 8), o),
                 lambda: moe.linear(big(1, n), big(8, n)), lambda: moe.linear(big(1, 8), big(n, 8)),
                 lambda: moe.linear_backward(big(1, n), big(1, 8), big(n, 8)),
                 lambda: moe.swiglu(big(1, 2 * n)), lambda: moe.swiglu_backward(big(1, n), big(1, 2 * n))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert moe.linear_backward_workspace_bytes(8, n, 8, BF, "silu", True) == 0


@pytest.mark.parametrize("call", [
    lambda t: moe.grouped_gemm(t(R, K), bf(E, N, K), offs()),
    lambda t: moe.grouped_gemm(bf(R, K), t(E, N, K), offs()),
    lambda t: moe.grouped_gemm_dgrad(t(R, N), bf(E, N, K), offs()),
    lambda t: moe.grouped_gemm_wgrad(bf(R, N), t(R, K), offs()),
    lambda t: moe.linear(bf(R, K), t(N, K)),
    lambda t: moe.linear(bf(R, K), bf(N, K), bias=t(N, dtype=torch.float32)),
    lambda t: moe.linear(bf(R, K), bf(N, K), residual=t(R, N)),
    lambda t: moe.linear_backward(bf(R, N), bf(R, K), t(N, K)),
    lambda t: moe.linear_backward(bf(R, N), bf(R, K), bf(N, K), preact=t(R, N), activation="silu"),
    lambda t: moe.swiglu(t(R, 2 * N)),
    lambda t: moe.swiglu(bf(R, 2 * N), row_w=t(R, dtype=torch.float32)),
    lambda t: moe.swiglu_backward(t(R, N), bf(R, 2 * N)),
])
def test_tensors_that_require_grad_are_refused_while_grad_mode_is_on(call):
    """The result would not require grad, and the gradient would be lost without a word."""
    def leaf(*s, dtype=BF):
        return torch.zeros(*s, dtype=dtype, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        call(leaf)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(leaf)
    with pytest.raises(ValueError, match="CUDA"):
        call(lambda *s, dtype=BF: leaf(*s, dtype=dtype).detach())
