"""Training operators around the AdamW parameters: embedding, layer norm, distillation.

Two layers.  The entry points (``embedding_forward`` and the like) are the C ABI's calls
without the ma_ prefix: tensors are checked, their pointers and the stream handed over, a
negative status raised as MuonAdamWError.  ``embedding``, ``layer_norm`` and ``distill_loss``
are the same operators for torch's autograd, so that ``loss.backward()`` runs the library's
kernels; ``embedding`` can hand its table gradient to a MuonAdamW in token form, which
``step()`` then applies without building the dense gradient.

Parameters and their gradients are fp32; activations fp32, fp16 or bf16.  Activation tensors
have contiguous rows (the last dimension) at any common row stride.  Work is enqueued on
``stream`` (the tensors' device's current stream when None); outputs and workspaces come from
torch's allocator.  A backward pass that is captured into a graph obeys torch's rule for
captured gradients: no eager autograd graph of the same parameters may be alive meanwhile.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import (_AdamWHParams, _check, _ptr, _require_f32_cuda, _scratch, _stream_handle, load)

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_BITS = {torch.int32: 32, torch.int64: 64}


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------
def _on(device):
    """Launches go to the tensors' device, whichever device is current."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _empty(shape, dtype, device, stream):
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and stream != torch.cuda.current_stream(device):
        t.record_stream(stream)
    return t


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _type(name, dtype) -> int:
    if dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16 (got {dtype})")
    return _DTYPES[dtype]


def _rows(name, t):
    """(rows, columns, row stride in values) of an activation tensor (..., columns)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    dim = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // dim if dim else 0), dim, max(dim, 1)
    try:
        v = t if t.dim() == 2 else t.view(-1, dim)
    except RuntimeError:
        raise ValueError(f"{name} must have rows of one common stride") from None
    n = v.shape[0]
    if dim > 1 and v.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    stride = v.stride(0) if n > 1 else max(dim, 1)
    if stride < dim:
        raise ValueError(f"{name} has overlapping rows")
    return n, dim, stride


def _ints(name, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if t.dtype not in _BITS:
        raise ValueError(f"{name} must be int32 or int64 (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _BITS[t.dtype]


def _vector(name, t, dim):
    if t is None:
        return
    _require_f32_cuda(name, t)
    if t.numel() != dim:
        raise ValueError(f"{name} must hold {dim} values (got {t.numel()})")


def _table(name, t):
    _require_f32_cuda(name, t)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a (rows, dim) table")
    return t.shape


def _workspace(workspace, need, device, stream):
    """(tensor or None, bytes): the caller's workspace, or one allocated for the call."""
    if workspace is None:
        return (_scratch(need, device, stream), need) if need else (None, 0)
    _same_device(device, workspace=workspace)
    return workspace, workspace.numel() * workspace.element_size()


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
def embedding_forward(table, tokens, *, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * table[tokens] (ma_embedding_forward): tokens int32 or int64 of any shape, the
    result tokens.shape + (dim,) in out_dtype (float32 when None) or written to `out`.  A
    token outside [0, rows) is padding: a zero row."""
    rows, dim = _table("table", table)
    bits = _ints("tokens", tokens)
    shape = tuple(tokens.shape) + (dim,)
    if out is None:
        out = _empty(shape, out_dtype or torch.float32, table.device, stream)
    elif tuple(out.shape) != shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be {shape} of {out_dtype or out.dtype}")
    _same_device(table.device, tokens=tokens, out=out)
    _, _, stride = _rows("out", out)
    with _on(table.device):
        _check(load().ma_embedding_forward(
            _ptr(table), rows, dim, _ptr(tokens), bits, tokens.numel(), scale, _ptr(out),
            _type("out", out.dtype), stride, _stream_handle(stream, table.device)))
    return out


def embedding_workspace_bytes(rows: int, dim: int, n: int) -> int:
    """Workspace of embedding_backward and adamw_step_embedding for n tokens."""
    return int(load().ma_embedding_workspace_bytes(int(rows), int(dim), int(n)))


def _token_rows(tokens, dout, dim):
    bits = _ints("tokens", tokens)
    n, cols, stride = _rows("dout", dout)
    if cols != dim or n != tokens.numel():
        raise ValueError(f"dout {tuple(dout.shape)} does not match {tokens.numel()} tokens of {dim}")
    return bits, n, stride, _type("dout", dout.dtype)


def embedding_backward(dout, tokens, rows: int, *, scale: float = 1.0, grad=None,
                       accumulate: bool = False, workspace=None, stream=None):
    """The (rows, dim) fp32 table gradient (ma_embedding_backward) of dout = tokens.shape +
    (dim,), into `grad` (allocated when None) or, with accumulate, added to it."""
    if accumulate and grad is None:
        raise ValueError("accumulate needs a grad to add to")
    rows, dim = int(rows), dout.shape[-1]
    bits, n, stride, dtype = _token_rows(tokens, dout, dim)
    device = dout.device
    if grad is None:
        grad = _empty((rows, dim), torch.float32, device, stream)
    elif tuple(_table("grad", grad)) != (rows, dim):
        raise ValueError(f"grad must be ({rows}, {dim})")
    _same_device(device, tokens=tokens, grad=grad)
    lib = load()
    with _on(device):
        ws, size = _workspace(workspace, lib.ma_embedding_workspace_bytes(rows, dim, n), device,
                              stream)
        _check(lib.ma_embedding_backward(
            _ptr(tokens), bits, n, _ptr(dout), dtype, stride, scale, _ptr(grad), rows, dim,
            int(bool(accumulate)), _ptr(ws), size, _stream_handle(stream, device)))
    return grad


def adamw_step_embedding(param, tokens, dout, exp_avg, exp_avg_sq, *, scale: float = 1.0, step: int,
                         lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                         weight_decay: float = 0.0, decoupled: bool = True,
                         cautious_wd: bool = False, workspace=None, stream=None) -> None:
    """One AdamW step of a (rows, dim) table (ma_adamw_step_embedding) with the gradient of
    embedding_backward(dout, tokens, rows, scale=scale), which is not materialised: bitwise
    adamw_step on that gradient."""
    rows, dim = _table("param", param)
    for name, t in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if tuple(_table(name, t)) != (rows, dim):
            raise ValueError(f"{name} must be ({rows}, {dim})")
    bits, n, stride, dtype = _token_rows(tokens, dout, dim)
    device = param.device
    _same_device(device, tokens=tokens, dout=dout, exp_avg=exp_avg, exp_avg_sq=exp_avg_sq)
    hp = _AdamWHParams(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                       step=int(step), decoupled=int(bool(decoupled)),
                       cautious_wd=int(bool(cautious_wd)))
    lib = load()
    with _on(device):
        ws, size = _workspace(workspace, lib.ma_embedding_workspace_bytes(rows, dim, n), device,
                              stream)
        _check(lib.ma_adamw_step_embedding(
            _ptr(param), _ptr(exp_avg), _ptr(exp_avg_sq), rows, dim, _ptr(tokens), bits, n,
            _ptr(dout), dtype, stride, scale, ctypes.byref(hp), _ptr(ws), size,
            _stream_handle(stream, device)))


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-5, out=None, stream=None):
    """(y, mean, rstd) of ma_layer_norm_forward over x's last dimension.  weight and bias:
    fp32 vectors or None; y has x's type; mean and rstd (x.shape[:-1], fp32) are the
    backward pass's inputs."""
    n, dim, stride = _rows("x", x)
    _vector("weight", weight, dim)
    _vector("bias", bias, dim)
    dtype, device = _type("x", x.dtype), x.device
    if out is None:
        out = _empty(x.shape, x.dtype, device, stream)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have x's shape and type")
    _, _, out_stride = _rows("out", out)
    _same_device(device, weight=weight, bias=bias, out=out)
    mean = _empty(x.shape[:-1], torch.float32, device, stream)
    rstd = _empty(x.shape[:-1], torch.float32, device, stream)
    with _on(device):
        _check(load().ma_layer_norm_forward(
            _ptr(x), dtype, stride, n, dim, _ptr(weight), _ptr(bias), eps, _ptr(out), out_stride,
            _ptr(mean), _ptr(rstd), _stream_handle(stream, device)))
    return out, mean, rstd


def layer_norm_workspace_bytes(n: int, dim: int) -> int:
    """Workspace of layer_norm_backward for n rows."""
    return int(load().ma_layer_norm_workspace_bytes(int(n), int(dim)))


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, weight_grad: bool = True,
                        bias_grad: bool = True, dweight=None, dbias=None, accumulate: bool = False,
                        workspace=None, stream=None):
    """(dx, dweight, dbias) of ma_layer_norm_backward.  weight_grad / bias_grad False leaves
    that one out (None).  dweight, dbias: fp32 vectors to write, or with accumulate to add to
    (allocated when None)."""
    n, dim, x_stride = _rows("x", x)
    dn, ddim, dy_stride = _rows("dy", dy)
    if (dn, ddim) != (n, dim) or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    _vector("weight", weight, dim)
    _vector("mean", mean, n)
    _vector("rstd", rstd, n)
    device = x.device
    for name, t, wanted in (("dweight", dweight, weight_grad), ("dbias", dbias, bias_grad)):
        _vector(name, t, dim)
        if t is not None and not wanted:
            raise ValueError(f"{name} is given but not wanted")
        if accumulate and wanted and t is None:
            raise ValueError(f"accumulate needs a {name} to add to")
    dx = _empty(x.shape, x.dtype, device, stream)
    if weight_grad and dweight is None:
        dweight = _empty(dim, torch.float32, device, stream)
    if bias_grad and dbias is None:
        dbias = _empty(dim, torch.float32, device, stream)
    _same_device(device, dy=dy, mean=mean, rstd=rstd, weight=weight, dweight=dweight, dbias=dbias)
    lib = load()
    with _on(device):
        need = lib.ma_layer_norm_workspace_bytes(n, dim) if weight_grad or bias_grad else 0
        ws, size = _workspace(workspace, need, device, stream)
        _check(lib.ma_layer_norm_backward(
            _ptr(dy), dy_stride, _ptr(x), x_stride, _type("x", x.dtype), n, dim, _ptr(weight),
            _ptr(mean), _ptr(rstd), _ptr(dx), max(dim, 1), _ptr(dweight), _ptr(dbias),
            int(bool(accumulate)), _ptr(ws), size, _stream_handle(stream, device)))
    return dx, dweight, dbias


# --------------------------------------------------------------------------
# distillation
# --------------------------------------------------------------------------
def _distill(logits, teacher, ids, temperature):
    """The leading arguments shared by the three calls, and (rows, vocab)."""
    n, vocab, stride = _rows("logits", logits)
    if not isinstance(teacher, torch.Tensor) or teacher.shape[:-1] != logits.shape[:-1] \
            or not teacher.is_contiguous():
        raise ValueError("teacher must be contiguous with the logits' leading dimensions")
    bits = _ints("ids", ids)
    if ids.shape != teacher.shape:
        raise ValueError("ids must have the teacher's shape")
    _same_device(logits.device, teacher=teacher, ids=ids)
    return (_ptr(logits), _type("logits", logits.dtype), stride, n, vocab, _ptr(teacher),
            _type("teacher", teacher.dtype), _ptr(ids), bits, teacher.shape[-1],
            float(temperature)), n


def _dlogits(logits, dlogits, stream):
    if dlogits is None:
        return _empty(logits.shape, logits.dtype, logits.device, stream)
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must have the logits' shape and type")
    _same_device(logits.device, dlogits=dlogits)
    return dlogits


def distill_forward(logits, teacher, ids, *, temperature: float = 1.0, stream=None):
    """(loss, stats) of ma_distill_forward: the Kullback-Leibler divergence, times
    temperature^2, of each row of logits (..., vocab) from the teacher's top logits (..., top)
    at the vocabulary places ids.  loss has the leading dimensions; stats (..., 2) is the
    backward pass's input."""
    args, _ = _distill(logits, teacher, ids, temperature)
    device = logits.device
    loss = _empty(logits.shape[:-1], torch.float32, device, stream)
    stats = _empty(tuple(logits.shape[:-1]) + (2,), torch.float32, device, stream)
    with _on(device):
        _check(load().ma_distill_forward(*args, _ptr(loss), _ptr(stats),
                                         _stream_handle(stream, device)))
    return loss, stats


def distill_backward(logits, teacher, ids, stats, row_weight, *, temperature: float = 1.0,
                     dlogits=None, stream=None):
    """The gradient of sum row_weight * loss by the logits (ma_distill_backward), into
    `dlogits` (allocated when None; may be `logits` itself)."""
    args, n = _distill(logits, teacher, ids, temperature)
    device = logits.device
    _vector("stats", stats, 2 * n)
    _vector("row_weight", row_weight, n)
    _same_device(device, stats=stats, row_weight=row_weight)
    dlogits = _dlogits(logits, dlogits, stream)
    _, _, stride = _rows("dlogits", dlogits)
    with _on(device):
        _check(load().ma_distill_backward(*args, _ptr(stats), _ptr(row_weight), _ptr(dlogits),
                                          stride, _stream_handle(stream, device)))
    return dlogits


def distill_loss_grad(logits, teacher, ids, row_weight, *, temperature: float = 1.0, dlogits=None,
                      stream=None):
    """(loss, dlogits) in one pass (ma_distill_loss_grad), for a row_weight known beforehand:
    the values of distill_forward and distill_backward."""
    args, n = _distill(logits, teacher, ids, temperature)
    device = logits.device
    _vector("row_weight", row_weight, n)
    _same_device(device, row_weight=row_weight)
    loss = _empty(logits.shape[:-1], torch.float32, device, stream)
    dlogits = _dlogits(logits, dlogits, stream)
    _, _, stride = _rows("dlogits", dlogits)
    with _on(device):
        _check(load().ma_distill_loss_grad(*args, _ptr(row_weight), _ptr(loss), _ptr(dlogits),
                                           stride, _stream_handle(stream, device)))
    return loss, dlogits


# --------------------------------------------------------------------------
# the same for autograd
# --------------------------------------------------------------------------
def _rowed(t):
    """t itself where its rows have one stride, else a contiguous copy (the expanded
    gradients that autograd makes for sums)."""
    try:
        _rows("gradient", t)
        return t
    except ValueError:
        return t.contiguous()


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, out_dtype, optimizer):
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.scale = table.shape[0], scale
        ctx.optimizer, ctx.table = optimizer, table if optimizer is not None else None
        return embedding_forward(table, tokens, scale=scale, out_dtype=out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        if not ctx.needs_input_grad[1]:
            return None, None, None, None, None
        (tokens,), dout = ctx.saved_tensors, _rowed(dout)
        if ctx.optimizer is not None:
            ctx.optimizer.add_token_gradient(ctx.table, tokens, dout, ctx.scale)
            return None, None, None, None, None
        return None, embedding_backward(dout, tokens, ctx.rows, scale=ctx.scale), None, None, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(_rowed(dy), x, mean, rstd, weight,
                                         weight_grad=ctx.needs_input_grad[1],
                                         bias_grad=ctx.needs_input_grad[2])
        return dx, dw, db, None


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher, ids, temperature):
        loss, stats = distill_forward(logits, teacher, ids, temperature=temperature)
        ctx.save_for_backward(logits, teacher, ids, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return None, None, None, None
        logits, teacher, ids, stats = ctx.saved_tensors
        return distill_backward(logits, teacher, ids, stats, dloss.contiguous(),
                                temperature=ctx.temperature), None, None, None


def embedding(tokens, table, *, scale: float = 1.0, out_dtype=None, optimizer=None):
    """scale * table[tokens], differentiable by the fp32 table; a token outside the table is
    padding (zero row, no gradient).  With `optimizer` (the MuonAdamW that holds the table in
    an "adamw" group) the backward pass sets no table.grad: it hands the tokens and output
    gradients to optimizer.add_token_gradient, and the next step() applies them."""
    return _Embedding.apply(tokens, table, float(scale), out_dtype, optimizer)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm over the last dimension with fp32 weight and bias (or None),
    differentiable by all three."""
    return _LayerNorm.apply(x, weight, bias, float(eps))


def distill_loss(logits, teacher, ids, *, temperature: float = 1.0):
    """The distillation loss of each row (see distill_forward), differentiable by the logits;
    the teacher is constant."""
    return _DistillLoss.apply(logits, teacher, ids, float(temperature))
