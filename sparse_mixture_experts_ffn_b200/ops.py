"""Operators next to the MoE layer (C ABI in ``include/moe_ops.h``): matrix products grouped by
expert, a linear layer with a fused epilogue, and the gated activation, each with its gradient.

Argument checking and marshalling only, as for the layer itself: the tensors' shapes, types and
devices are checked here (ValueError, before anything is launched), every sum runs in the
library's CUDA kernels, and there is no fallback.  The calls run on the tensors' device, on its
current stream unless ``stream`` is given (results not passed in are then allocated on that stream,
and using them on another one needs the usual ordering); they record no autograd graph: a training
loop calls the gradients itself, and a tensor that requires grad is refused (ValueError) while grad
mode is on, since its gradient would be lost.  A result that overlaps an input or another result is refused
(MoEError), but for ``linear``'s y, which may be its residual.

    r = moe_layer_forward(x, W_router, ...)[1]          # routing: r.offsets, r.perm, r.topk_w
    xp = x[r.perm.long() // top_k]
    gu = grouped_gemm(xp, W_gate_up, r.offsets)         # [T k, 2 I]
    h = swiglu(gu, row_w=w)                             # [T k, I]
    o = grouped_gemm(h, W_down, r.offsets)              # [T k, H]
    ...
    dh = grouped_gemm_dgrad(do, W_down, r.offsets)
    dW_down = grouped_gemm_wgrad(do, h, r.offsets)
    dgu, dw = swiglu_backward(dh, gu, row_w=w)
"""
from __future__ import annotations

import ctypes

from . import MOE_BF16, MOE_F32, MOE_OK, MoEError, load_library

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

EXPORTED = ("moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_linear",
            "moe_linear_backward_workspace_bytes", "moe_linear_backward", "moe_swiglu", "moe_swiglu_backward",
            "moe_ops_check_status")


class MoEGemmShape(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def declare(lib):
    """Argument types of the library's operator entry points."""
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    S = ctypes.POINTER(MoEGemmShape)
    for name, args in (("moe_grouped_gemm", [S, P, P, P, P, P]), ("moe_grouped_gemm_dgrad", [S, P, P, P, P, P]),
                       ("moe_grouped_gemm_wgrad", [S, P, P, P, P, P]),
                       ("moe_linear", [S, P, P, P, P, I32, P, P, P]),
                       ("moe_linear_backward", [S, P, P, P, P, I32, P, P, P, P, ctypes.c_size_t, P]),
                       ("moe_swiglu", [I64, I32, I32, P, P, F, P, P]),
                       ("moe_swiglu_backward", [I64, I32, I32, P, P, P, F, P, P, P]),
                       ("moe_ops_check_status", [P])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_linear_backward_workspace_bytes.argtypes = [S, I32, I32]
    lib.moe_linear_backward_workspace_bytes.restype = ctypes.c_size_t


_DTYPE_CODES = {}  # torch dtype -> moe_dtype, filled at the first call (torch is imported late)


def _dtype_code(name, t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        if not _DTYPE_CODES:
            import torch
            _DTYPE_CODES.update({torch.bfloat16: MOE_BF16, torch.float32: MOE_F32})
            return _dtype_code(name, t)
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return code


def _check(name, t, dtype, shape, device):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(R, N, K, E, code):
    if max(N, K, E) >= 1 << 31:  # a C field would wrap
        raise ValueError(f"sizes must be below 2^31, got N {N}, K {K}, E {E}")
    return MoEGemmShape(R, N, K, E, code)


def _no_graph(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            import torch
            if torch.is_grad_enabled():
                raise ValueError("a tensor requires grad, and these calls record no graph: call them under "
                                 "torch.no_grad() or on detached tensors, and the gradient functions yourself")


def _cuda(t):
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors (the operators run only on the GPU)")


def _call(entry, device, stream, *args):
    """Call ``entry`` with the stream's handle as its last argument, with ``device`` current."""
    import torch
    index = device.index
    # the current stream's handle without the Stream object around it: 2 us less a call
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    fn = getattr(load_library(), entry)
    if index == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != MOE_OK:
        raise MoEError(rc, entry)


def _new(like, shape, stream, dtype=None):
    """An uninitialised tensor on ``like``'s device, from the memory of the stream that will write it: the
    allocator may hand out memory that earlier work of the *current* stream still uses."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _grouped(entry, rows, W, offsets, out, out_name, stream, cols):
    """The two products against the experts' weights: rows [R, *] and W [E, N, K]."""
    import torch
    if rows.dim() != 2 or W.dim() != 3:
        raise ValueError("the row operand must be 2-D and W [E, N, K]")
    code = _dtype_code("the row operand", rows)
    R = rows.shape[0]
    E, N, K = W.shape
    dev = rows.device
    _check("the row operand", rows, rows.dtype, (R, K if cols == "N" else N), dev)
    _check("W", W, rows.dtype, (E, N, K), dev)
    _check("offsets", offsets, torch.int32, (E + 1,), dev)
    sizes = _shape(R, N, K, E, code)
    shape = (R, N if cols == "N" else K)
    if out is not None:
        _check(out_name, out, rows.dtype, shape, dev)
    _no_graph(rows, W)
    _cuda(rows)
    if out is None:
        out = _new(rows, shape, stream)
    _call(entry, dev, stream, sizes, rows.data_ptr(), W.data_ptr(), offsets.data_ptr(),
          out.data_ptr())
    return out


def grouped_gemm(x, W, offsets, *, y=None, stream=None):
    """y[r] = x[r] W[e]^T for the rows offsets[e] <= r < offsets[e + 1] of each expert e.

    x [R, K], W [E, N, K], offsets [E + 1] int32 on the device (non-decreasing, within
    [0, R]; ``Routing.offsets``), y [R, N]; bf16 (N and K multiples of 8) or fp32.  Rows
    outside all groups are not written: those of a new y are uninitialised, those of a given
    y stay as they are.  Offsets out of range make their expert empty and are reported by
    ``ops_check_status``.
    """
    return _grouped("moe_grouped_gemm", x, W, offsets, y, "y", stream, "N")


def grouped_gemm_dgrad(dy, W, offsets, *, dx=None, stream=None):
    """dx[r] = dy[r] W[e], the gradient of ``grouped_gemm``'s x: dy [R, N], W [E, N, K], dx
    [R, K]; rows outside all groups as for ``grouped_gemm``."""
    return _grouped("moe_grouped_gemm_dgrad", dy, W, offsets, dx, "dx", stream, "K")


def grouped_gemm_wgrad(dy, x, offsets, *, dW=None, stream=None):
    """dW[e] = sum over the rows r of expert e of dy[r]^T x[r], the gradient of
    ``grouped_gemm``'s W: dy [R, N], x [R, K], offsets [E + 1], dW [E, N, K] (written whole;
    zero for an expert without rows)."""
    import torch
    if dy.dim() != 2 or x.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("dy and x must be 2-D and offsets [E + 1]")
    code = _dtype_code("dy", dy)
    (R, N), K, E = dy.shape, x.shape[1], offsets.shape[0] - 1
    sizes = _shape(R, N, K, E, code)
    dev = dy.device
    _check("dy", dy, dy.dtype, (R, N), dev)
    _check("x", x, dy.dtype, (R, K), dev)
    _check("offsets", offsets, torch.int32, (E + 1,), dev)
    if dW is not None:
        _check("dW", dW, dy.dtype, (E, N, K), dev)
    _no_graph(dy, x)
    _cuda(dy)
    if dW is None:
        dW = _new(dy, (E, N, K), stream)
    _call("moe_grouped_gemm_wgrad", dev, stream, sizes, dy.data_ptr(), x.data_ptr(),
          offsets.data_ptr(), dW.data_ptr())
    return dW


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return code


def linear(x, W, *, bias=None, activation="none", residual=None, save_preact=False, y=None, preact=None, stream=None):
    """y = act(x W^T + bias) + residual, in one kernel.

    x [R, K], W [N, K], bias fp32 [N], residual and y [R, N] (y may be the residual itself);
    bf16 (N and K multiples of 8) or fp32.  activation: "none", "relu", "silu", "gelu" (error
    function) or "gelu_tanh".  Returns y, or with ``save_preact`` (or a given ``preact``
    [R, N]) the pair (y, x W^T + bias) that ``linear_backward`` needs.
    """
    import torch
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x must be [R, K] and W [N, K]")
    code = _dtype_code("x", x)
    act = _activation(activation)
    (R, K), N = x.shape, W.shape[0]
    sizes = _shape(R, N, K, 1, code)
    dev, dt = x.device, x.dtype
    _check("x", x, dt, (R, K), dev)
    _check("W", W, dt, (N, K), dev)
    if bias is not None:
        _check("bias", bias, torch.float32, (N,), dev)
    if residual is not None:
        _check("residual", residual, dt, (R, N), dev)
    if y is not None:
        _check("y", y, dt, (R, N), dev)
    if preact is not None:
        _check("preact", preact, dt, (R, N), dev)
    _no_graph(x, W, bias, residual)
    _cuda(x)
    if y is None:
        y = _new(x, (R, N), stream)
    if preact is None and save_preact:
        preact = _new(x, (R, N), stream)
    _call("moe_linear", dev, stream, sizes, x.data_ptr(), W.data_ptr(), _ptr(bias),
          _ptr(residual), act, y.data_ptr(), _ptr(preact))
    return y if preact is None else (y, preact)


def linear_backward(dy, x, W, *, preact=None, activation="none", input_grad=True, weight_grad=True, bias_grad=False,
                    dx=None, dW=None, dbias=None, workspace=None, stream=None):
    """Gradients of ``linear`` for the gradient dy [R, N] of its y: (dx, dW, dbias).

    dz = dy act'(preact); dx [R, K] = dz W, dW [N, K] = dz^T x, dbias fp32 [N] = sum of dz
    over the rows.  A gradient that is not wanted (``input_grad``, ``weight_grad``,
    ``bias_grad``) comes back as None; the residual's gradient is dy itself.  ``preact`` is
    the pre-activation that ``linear`` returned (not needed with activation "none").
    workspace: uint8 of at least ``linear_backward_workspace_bytes``, else one is allocated.
    """
    import torch
    if dy.dim() != 2 or x.dim() != 2 or W.dim() != 2:
        raise ValueError("dy must be [R, N], x [R, K] and W [N, K]")
    code = _dtype_code("dy", dy)
    act = _activation(activation)
    (R, N), K = dy.shape, W.shape[1]
    sizes = _shape(R, N, K, 1, code)
    dev, dt = dy.device, dy.dtype
    _check("dy", dy, dt, (R, N), dev)
    _check("x", x, dt, (R, K), dev)
    _check("W", W, dt, (N, K), dev)
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        _check("preact", preact, dt, (R, N), dev)
    else:
        preact = None
    for name, t, want, tdt, shape in (("dx", dx, input_grad, dt, (R, K)), ("dW", dW, weight_grad, dt, (N, K)),
                                      ("dbias", dbias, bias_grad, torch.float32, (N,))):
        if t is not None:
            if not want:
                raise ValueError(f"{name} is given but not asked for")
            _check(name, t, tdt, shape, dev)
    if workspace is not None and (workspace.device != dev or workspace.dtype != torch.uint8
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on dy's device")
    _no_graph(dy, x, W, preact)
    _cuda(dy)
    if input_grad and dx is None:
        dx = _new(dy, (R, K), stream)
    if weight_grad and dW is None:
        dW = _new(dy, (N, K), stream)
    if bias_grad and dbias is None:
        dbias = _new(dy, (N,), stream, torch.float32)
    nbytes = 0
    if workspace is not None:
        nbytes = workspace.numel()
    elif act or bias_grad:
        nbytes = load_library().moe_linear_backward_workspace_bytes(sizes, act, bool(bias_grad))
        workspace = _new(dy, (nbytes,), stream, torch.uint8) if nbytes else None
    _call("moe_linear_backward", dev, stream, sizes, dy.data_ptr(), x.data_ptr(), W.data_ptr(), _ptr(preact), act,
          _ptr(dx), _ptr(dW), _ptr(dbias), _ptr(workspace), nbytes)
    return dx, dW, dbias


def linear_backward_workspace_bytes(R, N, K, dtype, activation="none", bias_grad=False) -> int:
    """Workspace of ``linear_backward`` in bytes (0: none, or sizes that it does not take)."""
    import torch
    code = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}.get(dtype, -1)
    if max(N, K) >= 1 << 31:
        return 0
    return int(load_library().moe_linear_backward_workspace_bytes(_shape(R, N, K, 1, code),
                                                                  _activation(activation), bool(bias_grad)))


def _swiglu_args(gate_up, row_w, limit):
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise ValueError("gate_up must be [R, 2 I]")
    code = _dtype_code("gate_up", gate_up)
    R, I = gate_up.shape[0], gate_up.shape[1] // 2
    dev = gate_up.device
    if not gate_up.is_contiguous():
        raise ValueError("gate_up must be contiguous")
    if I >= 1 << 31:
        raise ValueError(f"sizes must be below 2^31, got I {I}")
    if row_w is not None:
        import torch
        _check("row_w", row_w, torch.float32, (R,), dev)
    limit = float(limit)
    if not 0.0 <= limit < float("inf"):
        raise ValueError(f"limit must be finite and >= 0, got {limit}")
    return code, R, I, dev, limit


def swiglu(gate_up, *, row_w=None, limit=0.0, h=None, stream=None):
    """h[r] = row_w[r] silu(min(gate, limit)) clamp(up, -limit, limit) on rows [gate | up].

    gate_up [R, 2 I] as ``grouped_gemm`` gives it for W_gate_up, row_w fp32 [R] (the routing
    weight) or None, h [R, I]; limit 0 is none.  bf16 (I a multiple of 8) or fp32.
    """
    code, R, I, dev, limit = _swiglu_args(gate_up, row_w, limit)
    if h is not None:
        _check("h", h, gate_up.dtype, (R, I), dev)
    _no_graph(gate_up, row_w)
    _cuda(gate_up)
    if h is None:
        h = _new(gate_up, (R, I), stream)
    _call("moe_swiglu", dev, stream, R, I, code, gate_up.data_ptr(), _ptr(row_w), limit, h.data_ptr())
    return h


def swiglu_backward(dh, gate_up, *, row_w=None, limit=0.0, d_gate_up=None, d_row_w=None, stream=None):
    """Gradients of ``swiglu`` for the gradient dh [R, I] of h: (d_gate_up [R, 2 I], d_row_w fp32
    [R], None without row_w).  The gradient passes where gate <= limit and |up| <= limit."""
    import torch
    code, R, I, dev, limit = _swiglu_args(gate_up, row_w, limit)
    _check("dh", dh, gate_up.dtype, (R, I), dev)
    if d_gate_up is not None:
        _check("d_gate_up", d_gate_up, gate_up.dtype, (R, 2 * I), dev)
    if d_row_w is not None:
        if row_w is None:
            raise ValueError("d_row_w is given without row_w")
        _check("d_row_w", d_row_w, torch.float32, (R,), dev)
    _no_graph(dh, gate_up, row_w)
    _cuda(gate_up)
    if d_gate_up is None:
        d_gate_up = _new(gate_up, (R, 2 * I), stream)
    if row_w is not None and d_row_w is None:
        d_row_w = _new(gate_up, (R,), stream, torch.float32)
    _call("moe_swiglu_backward", dev, stream, R, I, code, dh.data_ptr(), gate_up.data_ptr(), _ptr(row_w), limit,
          d_gate_up.data_ptr(), _ptr(d_row_w))
    return d_gate_up, d_row_w


def ops_check_status(device=None, stream=None) -> int:
    """Synchronise the stream and return, then clear, the device's status word of these
    operators: the first error recorded on the device since the last call (0 = MOE_OK)."""
    import torch
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream()
        return int(load_library().moe_ops_check_status(stream.cuda_stream))
