"""Training operators around the AdamW parameters: embedding, layer norm, distillation.

Two layers.  The entry points (``embedding_forward`` and the like) are the C ABI's calls
without the ma_ prefix: tensors are checked, their pointers and the stream handed over, a
negative status raised as MuonAdamWError.  ``embedding``, ``layer_norm`` and ``distill_loss``
are the same operators for torch's autograd, so that ``loss.backward()`` runs the library's
kernels; ``embedding`` can hand its table gradient to a MuonAdamW in token form, which
``step()`` then applies without building the dense gradient.

Parameters and their gradients are fp32; activations fp32, fp16 or bf16.  Activation tensors
have contiguous rows (the last dimension) at any common row stride; tokens, ids and teacher
lists any strides (they are copied where they are not contiguous).  Work is enqueued on
``stream`` (the tensors' device's current stream when None); outputs and workspaces come from
torch's allocator, from the memory of the stream that they are used on.  A call orders no
streams: with ``stream`` given, the caller has that stream wait for what makes the inputs, and
waits for it before using the outputs elsewhere.  A backward pass that is captured into a graph
obeys torch's rule for captured gradients: no eager autograd graph of the same parameters may be
alive meanwhile.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.graph import increment_version

from ._lib import _AdamWHParams, _check, _require_f32_cuda, _stream_handle, load

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_BITS = {torch.int32: 32, torch.int64: 64}


# --------------------------------------------------------------------------
# marshalling helpers.  Small calls are bound by this code, not by their kernels, so the
# checks touch each tensor once and the current stream is asked for its handle directly.
# --------------------------------------------------------------------------
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_functions: dict = {}


def _call(name, device, stream, *args):
    """The C call `name` with the stream's handle, on the tensors' device, whichever device
    is current."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream_handle(stream, device)
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load(), name)
    if device.index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status:
        _check(status)


def _record(stream, *tensors):
    """Work on a given stream: the tensors' memory is not handed out again before that stream
    is done with it, should the caller drop them."""
    for t in tensors:
        if t is not None and stream != torch.cuda.current_stream(t.device):
            t.record_stream(stream)


def record_use(*tensors):
    """Records tensors on their devices' current streams (see _record)."""
    for t in tensors:
        t.record_stream(torch.cuda.current_stream(t.device))


def _wrote(*tensors):
    """The caller's tensors that a call has written, by their addresses: their versions advance,
    so that autograd and MuonAdamW see that what they kept of them has changed."""
    increment_version([t for t in tensors if t is not None])


def _allocate(like, shape, dtype, stream):
    """A tensor on the device of `like` from the memory of `stream`: what the current stream has
    dropped may still be in use by work queued there, which `stream` does not wait for."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _empty(like, shape, dtype, stream):
    """An output: allocated on `stream`, and for the caller to use on the current one."""
    t = _allocate(like, shape, dtype, stream)
    if stream is not None:
        record_use(t)
    return t


def _like(t, stream):
    """A contiguous tensor of t's shape and type (the cheapest allocation there is)."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t, t.shape, t.dtype, stream)


def _tensor(name, t, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _type(name, dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16 (got {dtype})")
    return code


def _rows(name, t, device=None, anywhere=False):
    """(rows, columns, row stride in values) of an activation tensor (..., columns), on the GPU
    or anywhere."""
    if not anywhere:
        _tensor(name, t, device)
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


def _ints(name, t, device=None) -> int:
    _tensor(name, t, device)
    bits = _BITS.get(t.dtype)
    if bits is None:
        raise ValueError(f"{name} must be int32 or int64 (got {t.dtype})")
    return bits


def _contiguous(t, stream):
    """t, copied on the call's stream where it is not contiguous (to be kept for the call)."""
    if t.is_contiguous():
        return t
    with torch.cuda.stream(stream):
        return t.contiguous()


def _floats(name, t, count, device=None) -> int:
    """The address of an fp32 vector of `count` values; 0 for None."""
    if t is None:
        return 0
    _tensor(name, t, device)
    if t.dtype is not torch.float32 or not t.is_contiguous():
        _require_f32_cuda(name, t)
    if t.numel() != count:
        raise ValueError(f"{name} must hold {count} values (got {t.numel()})")
    return t.data_ptr()


def _table(name, t, device=None):
    _tensor(name, t, device)
    if t.dtype is not torch.float32 or not t.is_contiguous():
        _require_f32_cuda(name, t)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a (rows, dim) table")
    return t.shape


def _workspace(workspace, need, like, stream):
    """(the tensor to keep, address, bytes) of the caller's workspace, or of one allocated
    for the call."""
    if workspace is None:
        if not need:
            return None, 0, 0
        workspace = _allocate(like, need, torch.uint8, stream)
    else:
        _tensor("workspace", workspace, like.device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=256)
def embedding_workspace_bytes(rows: int, dim: int, n: int) -> int:
    """Workspace of embedding_backward and adamw_step_embedding for n tokens."""
    return int(load().ma_embedding_workspace_bytes(int(rows), int(dim), int(n)))


@functools.lru_cache(maxsize=256)
def layer_norm_workspace_bytes(n: int, dim: int) -> int:
    """Workspace of layer_norm_backward for n rows."""
    return int(load().ma_layer_norm_workspace_bytes(int(n), int(dim)))


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
def embedding_forward(table, tokens, *, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * table[tokens] (ma_embedding_forward): tokens int32 or int64 of any shape, the
    result tokens.shape + (dim,) in out_dtype (float32 when None) or written to `out`.  A
    token outside [0, rows) is padding: a zero row."""
    rows, dim = _table("table", table)
    device = table.device
    bits = _ints("tokens", tokens, device)
    shape, given = tokens.shape + (dim,), out
    at = tokens if tokens.is_contiguous() else _contiguous(tokens, stream)
    if out is None:
        out, stride = _empty(table, shape, out_dtype or torch.float32, stream), dim
    else:
        _tensor("out", out, device)
        if out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be {tuple(shape)} of {out_dtype or out.dtype}")
        _, _, stride = _rows("out", out, device)
    _call("ma_embedding_forward", device, stream, table.data_ptr(), rows, dim, at.data_ptr(),
          bits, tokens.numel(), scale, out.data_ptr(), _type("out", out.dtype), stride)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, table, tokens, out)
    return out


def _token_rows(tokens, dout, dim=None, device=None):
    n, cols, stride = _rows("dout", dout, device)
    bits = _ints("tokens", tokens, dout.device)
    if (dim is not None and cols != dim) or n != tokens.numel():
        raise ValueError(f"dout {tuple(dout.shape)} does not match {tokens.numel()} tokens of {dim or cols}")
    return bits, n, stride, _type("dout", dout.dtype)


def embedding_backward(dout, tokens, rows: int, *, scale: float = 1.0, grad=None,
                       accumulate: bool = False, workspace=None, stream=None):
    """The (rows, dim) fp32 table gradient (ma_embedding_backward) of dout = tokens.shape +
    (dim,), into `grad` (allocated when None) or, with accumulate, added to it."""
    if accumulate and grad is None:
        raise ValueError("accumulate needs a grad to add to")
    bits, n, stride, dtype = _token_rows(tokens, dout)
    rows, dim, device = int(rows), dout.shape[-1], dout.device
    given = grad
    if grad is None:
        grad = _empty(dout, (rows, dim), torch.float32, stream)
    elif tuple(_table("grad", grad, device)) != (rows, dim):
        raise ValueError(f"grad must be ({rows}, {dim})")
    need = embedding_workspace_bytes(rows, dim, n)
    _keep, ws, size = _workspace(workspace, need, dout, stream)
    at = tokens if tokens.is_contiguous() else _contiguous(tokens, stream)
    _call("ma_embedding_backward", device, stream, at.data_ptr(), bits, n, dout.data_ptr(),
          dtype, stride, scale, grad.data_ptr(), rows, dim, int(bool(accumulate)), ws, size)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, tokens, dout, grad, _keep)
    return grad


def adamw_step_embedding(param, tokens, dout, exp_avg, exp_avg_sq, *, scale: float = 1.0, step: int,
                         lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                         weight_decay: float = 0.0, decoupled: bool = True,
                         cautious_wd: bool = False, workspace=None, stream=None) -> None:
    """One AdamW step of a (rows, dim) table (ma_adamw_step_embedding) with the gradient of
    embedding_backward(dout, tokens, rows, scale=scale), which is not materialised: bitwise
    adamw_step on that gradient."""
    rows, dim = _table("param", param)
    device = param.device
    if _table("exp_avg", exp_avg, device) != param.shape or \
            _table("exp_avg_sq", exp_avg_sq, device) != param.shape:
        raise ValueError(f"exp_avg and exp_avg_sq must be ({rows}, {dim})")
    bits, n, stride, dtype = _token_rows(tokens, dout, dim, device)
    hp = _AdamWHParams(lr, beta1, beta2, eps, weight_decay, int(step), int(bool(decoupled)),
                       int(bool(cautious_wd)))
    need = embedding_workspace_bytes(rows, dim, n)
    _keep, ws, size = _workspace(workspace, need, param, stream)
    at = tokens if tokens.is_contiguous() else _contiguous(tokens, stream)
    _call("ma_adamw_step_embedding", device, stream, param.data_ptr(), exp_avg.data_ptr(),
          exp_avg_sq.data_ptr(), rows, dim, at.data_ptr(), bits, n, dout.data_ptr(), dtype,
          stride, scale, ctypes.byref(hp), ws, size)
    increment_version((param, exp_avg, exp_avg_sq))
    if stream is not None:
        _record(stream, param, exp_avg, exp_avg_sq, tokens, dout, _keep)


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-5, out=None, stream=None):
    """(y, mean, rstd) of ma_layer_norm_forward over x's last dimension.  weight and bias:
    fp32 vectors or None; y has x's type; mean and rstd (x.shape[:-1], fp32) are the
    backward pass's inputs."""
    n, dim, stride = _rows("x", x)
    dtype, device = _type("x", x.dtype), x.device
    w, b = _floats("weight", weight, dim, device), _floats("bias", bias, dim, device)
    given = out
    if out is None:
        out, out_stride = _like(x, stream), max(dim, 1)
    else:
        _tensor("out", out, device)
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have x's shape and type")
        _, _, out_stride = _rows("out", out, device)
    mean = _empty(x, x.shape[:-1], torch.float32, stream)
    rstd = _like(mean, stream)
    _call("ma_layer_norm_forward", device, stream, x.data_ptr(), dtype, stride, n, dim, w, b, eps,
          out.data_ptr(), out_stride, mean.data_ptr(), rstd.data_ptr())
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, x, weight, bias, out)
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, weight_grad: bool = True,
                        bias_grad: bool = True, dweight=None, dbias=None, accumulate: bool = False,
                        workspace=None, stream=None):
    """(dx, dweight, dbias) of ma_layer_norm_backward.  weight_grad / bias_grad False leaves
    that one out (None).  dweight, dbias: fp32 vectors to write, or with accumulate to add to
    (allocated when None)."""
    n, dim, x_stride = _rows("x", x)
    device = x.device
    dn, ddim, dy_stride = _rows("dy", dy, device)
    if dn != n or ddim != dim or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    if (dweight is not None and not weight_grad) or (dbias is not None and not bias_grad):
        raise ValueError("a gradient buffer is given for a gradient that is not wanted")
    if accumulate and ((weight_grad and dweight is None) or (bias_grad and dbias is None)):
        raise ValueError("accumulate needs the gradients to add to")
    given = (dweight, dbias)
    if weight_grad and dweight is None:
        dweight = _empty(x, dim, torch.float32, stream)
    if bias_grad and dbias is None:
        dbias = _like(dweight, stream) if weight_grad else _empty(x, dim, torch.float32, stream)
    dx = _like(x, stream)
    need = layer_norm_workspace_bytes(n, dim) if weight_grad or bias_grad else 0
    _keep, ws, size = _workspace(workspace, need, x, stream)
    _call("ma_layer_norm_backward", device, stream, dy.data_ptr(), dy_stride, x.data_ptr(), x_stride,
          _type("x", x.dtype), n, dim, _floats("weight", weight, dim, device),
          _floats("mean", mean, n, device), _floats("rstd", rstd, n, device), dx.data_ptr(),
          max(dim, 1), _floats("dweight", dweight, dim, device),
          _floats("dbias", dbias, dim, device), int(bool(accumulate)), ws, size)
    if given[0] is not None or given[1] is not None:
        _wrote(*given)
    if stream is not None:
        _record(stream, dy, x, mean, rstd, weight, dweight, dbias, _keep)
    return dx, dweight, dbias


# --------------------------------------------------------------------------
# distillation
# --------------------------------------------------------------------------
def _distill(logits, teacher, ids, temperature, stream):
    """The leading arguments shared by the three calls, the number of rows, and what the
    arguments' addresses need alive."""
    n, vocab, stride = _rows("logits", logits)
    _tensor("teacher", teacher, logits.device)
    if teacher.dim() != logits.dim() or teacher.shape[:-1] != logits.shape[:-1]:
        raise ValueError("teacher must have the logits' leading dimensions")
    bits = _ints("ids", ids, logits.device)
    if ids.shape != teacher.shape:
        raise ValueError("ids must have the teacher's shape")
    keep = teacher, ids = _contiguous(teacher, stream), _contiguous(ids, stream)
    return (logits.data_ptr(), _type("logits", logits.dtype), stride, n, vocab, teacher.data_ptr(),
            _type("teacher", teacher.dtype), ids.data_ptr(), bits, teacher.shape[-1],
            float(temperature)), n, keep


def _dlogits(logits, dlogits, stream):
    """(dlogits, row stride)"""
    if dlogits is None:
        return _like(logits, stream), logits.shape[-1]
    _tensor("dlogits", dlogits, logits.device)
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must have the logits' shape and type")
    return dlogits, _rows("dlogits", dlogits, logits.device)[2]


def distill_forward(logits, teacher, ids, *, temperature: float = 1.0, stream=None):
    """(loss, stats) of ma_distill_forward: the Kullback-Leibler divergence, times
    temperature^2, of each row of logits (..., vocab) from the teacher's top logits (..., top)
    at the vocabulary places ids.  loss has the leading dimensions; stats (..., 2) is the
    backward pass's input.  Positions without a target (the last ones of a batch of sequences)
    take ids of -1 and their logits stay where they are: loss and gradient are zero."""
    args, _, _keep = _distill(logits, teacher, ids, temperature, stream)
    loss = _empty(logits, logits.shape[:-1], torch.float32, stream)
    stats = _empty(logits, logits.shape[:-1] + (2,), torch.float32, stream)
    _call("ma_distill_forward", logits.device, stream, *args, loss.data_ptr(), stats.data_ptr())
    if stream is not None:
        _record(stream, logits, teacher, ids)
    return loss, stats


def distill_backward(logits, teacher, ids, stats, row_weight, *, temperature: float = 1.0,
                     dlogits=None, stream=None):
    """The gradient of sum row_weight * loss by the logits (ma_distill_backward), into
    `dlogits` (allocated when None; may be `logits` itself)."""
    args, n, _keep = _distill(logits, teacher, ids, temperature, stream)
    device = logits.device
    s, w = _floats("stats", stats, 2 * n, device), _floats("row_weight", row_weight, n, device)
    given = dlogits
    dlogits, stride = _dlogits(logits, dlogits, stream)
    _call("ma_distill_backward", device, stream, *args, s, w, dlogits.data_ptr(), stride)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, logits, teacher, ids, stats, row_weight, dlogits)
    return dlogits


def distill_loss_grad(logits, teacher, ids, row_weight, *, temperature: float = 1.0, dlogits=None,
                      stream=None):
    """(loss, dlogits) in one pass (ma_distill_loss_grad), for a row_weight known beforehand:
    the values of distill_forward and distill_backward."""
    args, n, _keep = _distill(logits, teacher, ids, temperature, stream)
    device = logits.device
    w = _floats("row_weight", row_weight, n, device)
    loss = _empty(logits, logits.shape[:-1], torch.float32, stream)
    given = dlogits
    dlogits, stride = _dlogits(logits, dlogits, stream)
    _call("ma_distill_loss_grad", device, stream, *args, w, loss.data_ptr(), dlogits.data_ptr(),
          stride)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, logits, teacher, ids, row_weight, dlogits)
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
        tokens = tokens.contiguous()
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
        ctx.shapes = [t if t is None else t.shape for t in (weight, bias)]
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(_rowed(dy), x, mean, rstd, weight,
                                         weight_grad=ctx.needs_input_grad[1],
                                         bias_grad=ctx.needs_input_grad[2])
        dw, db = (t if t is None else t.view(shape) for t, shape in zip((dw, db), ctx.shapes))
        return dx, dw, db, None


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher, ids, temperature):
        teacher, ids = teacher.contiguous(), ids.contiguous()
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
    gradients to optimizer.add_token_gradient, and the next step() applies them (not for loops
    that clip or unscale gradients in between: see there)."""
    if optimizer is not None:
        optimizer.check_token_parameter(table)
    return _Embedding.apply(tokens, table, float(scale), out_dtype, optimizer)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm over the last dimension with fp32 weight and bias (or None),
    differentiable by all three."""
    return _LayerNorm.apply(x, weight, bias, float(eps))


def distill_loss(logits, teacher, ids, *, temperature: float = 1.0):
    """The distillation loss of each row (see distill_forward), differentiable by the logits;
    the teacher is constant."""
    return _DistillLoss.apply(logits, teacher, ids, float(temperature))
