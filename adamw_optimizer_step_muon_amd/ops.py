"""Training operators around the AdamW parameters: embedding, layer norm, the norms around a
block, distillation, the LM head's cross entropy, and the AdamW step with moments in 8 bits.

Two layers.  The entry points (``embedding_forward`` and the like) are the C ABI's calls
without the ma_ prefix: tensors are checked, their pointers and the stream handed over, a
negative status raised as MuonAdamWError.  ``embedding``, ``layer_norm``, ``residual_norm``,
``distill_loss`` and ``head_loss`` are the same operators for torch's autograd, so that ``loss.backward()`` runs the library's
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
import struct

import torch
from torch.autograd.graph import increment_version

from ._lib import (_AdamWByteHParams, _AdamWByteSegment, _AdamWHParams, _check, _require_f32_cuda,
                   _ResidualNormGrads, _ResidualNormParams, _stream_handle, load)

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


def _address(t) -> int:
    return 0 if t is None else t.data_ptr()


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
# the norms around a block
# --------------------------------------------------------------------------
@functools.lru_cache(maxsize=256)
def residual_norm_workspace_bytes(n: int, dim: int) -> int:
    """Workspace of residual_norm_backward for n rows."""
    return int(load().ma_residual_norm_workspace_bytes(int(n), int(dim)))


def _residual_params(dim, device, weight, bias, post_norm, post_weight, post_bias, gate, scale, center, eps):
    if not post_norm and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias are for a call with post_norm")
    return _ResidualNormParams(
        _floats("post_weight", post_weight, dim, device), _floats("post_bias", post_bias, dim, device),
        _floats("gate", gate, dim, device), _floats("weight", weight, dim, device),
        _floats("bias", bias, dim, device), scale, eps, int(bool(post_norm)), int(bool(center)))


def _alike(name, t, like, device):
    """The row stride of a tensor of the shape and type of `like`."""
    _tensor(name, t, device)
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must have x's shape and type")
    return _rows(name, t, device)[2]


def residual_norm_forward(x, residual, weight=None, bias=None, *, post_norm: bool = True, post_weight=None,
                          post_bias=None, gate=None, scale: float = 1.0, center: bool = True,
                          eps: float = 1e-5, out=None, stream=None):
    """(out, y, stats) of ma_residual_norm_forward over x's last dimension: the residual stream
    behind a block with output x, out = residual + scale * gate * norm(x) (with post_norm False:
    of x itself), and y = norm(out), the next block's input.  The norms are layer norms with fp32
    gains and biases, or None; center False makes them root-mean-square norms.  gate: an fp32
    vector or None.  out and y have x's type (out may be given, also as the residual itself);
    stats (4, *x.shape[:-1], fp32) are the backward pass's input."""
    n, dim, x_stride = _rows("x", x)
    device, dtype = x.device, _type("x", x.dtype)
    residual_stride = _alike("residual", residual, x, device)
    params = _residual_params(dim, device, weight, bias, post_norm, post_weight, post_bias, gate, scale, center, eps)
    given = out
    if out is None:
        out, out_stride = _like(x, stream), max(dim, 1)
    else:
        out_stride = _alike("out", out, x, device)
    y = _like(x, stream)
    stats = _empty(x, (4,) + x.shape[:-1], torch.float32, stream)
    _call("ma_residual_norm_forward", device, stream, x.data_ptr(), x_stride, residual.data_ptr(), residual_stride,
          dtype, n, dim, ctypes.byref(params), out.data_ptr(), out_stride, y.data_ptr(), max(dim, 1), stats.data_ptr())
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, x, residual, weight, bias, post_weight, post_bias, gate, out)
    return out, y, stats


def residual_norm_backward(dout, dy, x, out, stats, weight=None, bias=None, *, post_norm: bool = True,
                           post_weight=None, post_bias=None, gate=None, scale: float = 1.0,
                           center: bool = True, param_grads=True, workspace=None, stream=None):
    """(dx, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate) of ma_residual_norm_backward;
    dout None means zeros.  A parameter that is None has no gradient (None); param_grads is True or
    False for all of them, or five truth values in the order of the result."""
    n, dim, x_stride = _rows("x", x)
    device, dtype = x.device, _type("x", x.dtype)
    dout_stride = dim if dout is None else _alike("dout", dout, x, device)
    dy_stride, out_stride = _alike("dy", dy, x, device), _alike("out", out, x, device)
    # (eps is in the statistics)
    params = _residual_params(dim, device, weight, bias, post_norm, post_weight, post_bias, gate, scale, center, 0.0)
    if isinstance(param_grads, bool):
        param_grads = (param_grads,) * 5
    grads = [None if t is None or not want else _empty(x, dim, torch.float32, stream)
             for t, want in zip((weight, bias, post_weight, post_bias, gate), param_grads)]
    at = [_address(t) for t in grads]
    dx = _like(x, stream)
    dresidual = _like(dx, stream)
    need = residual_norm_workspace_bytes(n, dim) if any(t is not None for t in grads) else 0
    _keep, ws, size = _workspace(workspace, need, x, stream)
    _call("ma_residual_norm_backward", device, stream, _address(dout), dout_stride, dy.data_ptr(), dy_stride,
          x.data_ptr(), x_stride, out.data_ptr(), out_stride, _floats("stats", stats, 4 * n, device), dtype, n, dim,
          ctypes.byref(params), ctypes.byref(_ResidualNormGrads(at[2], at[3], at[4], at[0], at[1])), dx.data_ptr(),
          max(dim, 1), dresidual.data_ptr(), max(dim, 1), ws, size)
    if stream is not None:
        _record(stream, dout, dy, x, out, stats, weight, bias, post_weight, post_bias, gate, _keep)
    return dx, dresidual, *grads


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
# the LM head's cross entropy
# --------------------------------------------------------------------------
_HEAD_CALLS = {"forward": 0, "backward": 2, "grad": 3}


@functools.lru_cache(maxsize=256)
def _head_workspace(dtype: int, n: int, dim: int, vocab: int, aligned: int, stride: int, calls: int) -> int:
    # of the weight's address only its alignment counts
    return int(load().ma_head_loss_workspace_bytes(dtype, n, dim, vocab, 256 + aligned, stride, calls))


def head_loss_workspace_bytes(hidden, weight, *, gradients: bool = True, call=None) -> int:
    """Workspace for any of the head loss calls on these tensors; gradients False: for the forward call;
    call "forward", "backward" or "grad": for that one alone."""
    if call is not None and call not in _HEAD_CALLS:
        raise ValueError(f"call must be one of {sorted(_HEAD_CALLS)} (got {call!r})")
    n, dim, _ = _rows("hidden", hidden, anywhere=True)
    vocab, _, stride = _rows("weight", weight, anywhere=True)
    return _head_workspace(_type("hidden", hidden.dtype), n, dim, vocab, weight.data_ptr() % 16, stride,
                           int(bool(gradients)) if call is None else _HEAD_CALLS[call])


def _head(hidden, weight, labels, call, workspace, stream):
    """The leading arguments shared by the three calls, the number of rows, the workspace, and
    what the arguments' addresses need alive."""
    n, dim, hidden_stride = _rows("hidden", hidden)
    device, dtype = hidden.device, _type("hidden", hidden.dtype)
    vocab, wdim, weight_stride = _rows("weight", weight, device)
    if weight.dim() != 2 or wdim != dim or weight.dtype != hidden.dtype:
        raise ValueError(f"weight must be (vocab, {dim}) of {hidden.dtype}")
    bits = _ints("labels", labels, device)
    if labels.shape != hidden.shape[:-1]:
        raise ValueError("labels must have the hidden states' leading dimensions")
    at = labels if labels.is_contiguous() else _contiguous(labels, stream)
    need = _head_workspace(dtype, n, dim, vocab, weight.data_ptr() % 16, weight_stride,
                           _HEAD_CALLS[call])
    keep, ws, size = _workspace(workspace, need, hidden, stream)
    return (hidden.data_ptr(), dtype, hidden_stride, n, dim, weight.data_ptr(), weight_stride, vocab, at.data_ptr(),
            bits), n, (ws, size), (keep, at)


def _head_gradients(hidden, weight, hidden_grad, weight_grad, dweight, accumulate, stream):
    """(dhidden, dweight, their arguments)"""
    if dweight is not None and not weight_grad:
        raise ValueError("a gradient buffer is given for a gradient that is not wanted")
    if accumulate and dweight is None and weight_grad:
        raise ValueError("accumulate needs a dweight to add to")
    dhidden = _like(hidden, stream) if hidden_grad else None
    stride = max(hidden.shape[-1], 1)
    dtype = _type("weight", weight.dtype)
    if dweight is not None:
        _tensor("dweight", dweight, hidden.device)
        if dweight.shape != weight.shape or dweight.dtype not in (torch.float32, weight.dtype):
            raise ValueError("dweight must have the weight's shape, and its type or float32")
        dtype, stride = _type("dweight", dweight.dtype), _rows("dweight", dweight, hidden.device)[2]
    elif weight_grad:
        dweight = _like(weight, stream)
    return dhidden, dweight, (_address(dhidden), max(hidden.shape[-1], 1), _address(dweight), dtype, stride,
                              int(bool(accumulate)))


def head_loss_forward(hidden, weight, labels, *, workspace=None, stream=None):
    """(loss, lse) of ma_head_loss_forward: the softmax cross entropy of labels (int32 or int64, the
    hidden states' leading dimensions) under the logits hidden (..., dim) @ weight (vocab, dim).T,
    which are not kept.  hidden and weight have one type; weight is the head in that type (see
    adamw_byte_step_multi's copies).  A label outside the vocabulary marks a row without a target:
    loss and lse 0.  lse, the logarithm of the sum of exponentials, is the backward pass's input."""
    args, _, space, _keep = _head(hidden, weight, labels, "forward", workspace, stream)
    loss = _empty(hidden, hidden.shape[:-1], torch.float32, stream)
    lse = _like(loss, stream)
    _call("ma_head_loss_forward", hidden.device, stream, *args, loss.data_ptr(), lse.data_ptr(), *space)
    if stream is not None:
        _record(stream, hidden, weight, labels, *_keep)
    return loss, lse


def head_loss_backward(hidden, weight, labels, lse, row_weight, *, hidden_grad: bool = True,
                       weight_grad: bool = True, dweight=None, accumulate: bool = False,
                       workspace=None, stream=None):
    """(dhidden, dweight) of ma_head_loss_backward: the gradients of sum row_weight * loss.  Either
    can be left out (None).  dweight has the weight's type, or is given: of that type, or float32
    and with accumulate added to.  The logits' gradients are rounded to the hidden type once."""
    args, n, space, _keep = _head(hidden, weight, labels, "backward", workspace, stream)
    device, given = hidden.device, dweight
    rows = _floats("lse", lse, n, device), _floats("row_weight", row_weight, n, device)
    dhidden, dweight, outs = _head_gradients(hidden, weight, hidden_grad, weight_grad, dweight, accumulate, stream)
    _call("ma_head_loss_backward", device, stream, *args, *rows, *outs, *space)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, hidden, weight, labels, lse, row_weight, given, *_keep)
    return dhidden, dweight


def head_loss_grad(hidden, weight, labels, row_weight, *, hidden_grad: bool = True, weight_grad: bool = True,
                   dweight=None, accumulate: bool = False, workspace=None, stream=None):
    """(loss, dhidden, dweight) in one call (ma_head_loss_grad), for a row_weight known beforehand."""
    args, n, space, _keep = _head(hidden, weight, labels, "grad", workspace, stream)
    device, given = hidden.device, dweight
    row = _floats("row_weight", row_weight, n, device)
    loss = _empty(hidden, hidden.shape[:-1], torch.float32, stream)
    dhidden, dweight, outs = _head_gradients(hidden, weight, hidden_grad, weight_grad, dweight, accumulate, stream)
    _call("ma_head_loss_grad", device, stream, *args, row, loss.data_ptr(), *outs, *space)
    if given is not None:
        _wrote(given)
    if stream is not None:
        _record(stream, hidden, weight, labels, row_weight, given, *_keep)
    return loss, dhidden, dweight


# --------------------------------------------------------------------------
# AdamW with both moments in 8 bits
# --------------------------------------------------------------------------
ADAMW_BYTE_BLOCK = 64  # elements that share a scale
_BYTE_SEGMENT = struct.Struct("=7Qq2i")  # _AdamWByteSegment
_HALVES = (torch.float16, torch.bfloat16)
_ADAMW_BYTE_STATE = (("exp_avg", torch.float8_e4m3fn, 1), ("exp_avg_scale", torch.float8_e8m0fnu, ADAMW_BYTE_BLOCK),
                 ("exp_avg_sq", torch.float8_e5m2, 1), ("exp_avg_sq_scale", torch.float8_e8m0fnu, ADAMW_BYTE_BLOCK))


def adamw_byte_state(param):
    """(exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale) of `param` before its first step:
    zeros in the parameter's shape (e4m3 and e5m2) and scales of one (e8m0), one per block of 64
    consecutive elements."""
    scale = torch.full((-(-param.numel() // ADAMW_BYTE_BLOCK),), 127, dtype=torch.uint8, device=param.device)
    scale = scale.view(torch.float8_e8m0fnu)
    zeros = torch.zeros(param.shape, dtype=torch.uint8, device=param.device)
    return (zeros.view(torch.float8_e4m3fn), scale,
            zeros.clone().view(torch.float8_e5m2), scale.view(torch.uint8).clone().view(torch.float8_e8m0fnu))


def adamw_byte_values(value, scale):
    """What a moment's 8-bit values and their blocks' scales stand for, in fp32."""
    flat = value.reshape(-1).float()
    return flat.mul_(scale.float().repeat_interleave(ADAMW_BYTE_BLOCK)[:flat.numel()]).view(value.shape)


def adamw_byte_step_multi(segments, *, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                      eps: float = 1e-8, weight_decay: float = 0.0, decoupled: bool = True,
                      cautious_wd: bool = False, seed: int = 0, stream=None) -> None:
    """One AdamW step over many tensors with their moments in 8 bits (ma_adamw_byte_step_multi).  A
    segment is (param, grad, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale) or, with one
    more entry, ..., copy): param contiguous fp32, grad fp32, fp16 or bf16, the moments as
    adamw_byte_state lays them out, and copy None or an fp16 or bf16 tensor that receives the stepped
    parameter.  `seed` numbers the roundings' random bits, together with `step`."""
    segments = list(segments)
    if not segments:
        return
    buf, written, at = bytearray(len(segments) * _BYTE_SEGMENT.size), [], 0
    device = None
    for i, seg in enumerate(segments):
        if len(seg) == 7:
            p, g, m, ms, v, vs, copy = seg
        elif len(seg) == 6:
            (p, g, m, ms, v, vs), copy = seg, None
        else:
            raise ValueError(f"segment {i} must hold 6 or 7 tensors")
        # the usual segment passes in as few looks at its tensors as there can be; the reasons
        # of the others are found by _refuse_byte_segment
        try:
            n, index = p.numel(), p.get_device()
            blocks = -(-n // ADAMW_BYTE_BLOCK)
            fine = (index >= 0 and (device is None or index == device.index)
                    and p.dtype is torch.float32 and p.is_contiguous()
                    and g.numel() == n and g.is_contiguous() and g.get_device() == index
                    and m.dtype is torch.float8_e4m3fn and m.numel() == n and m.is_contiguous() and m.get_device() == index
                    and v.dtype is torch.float8_e5m2 and v.numel() == n and v.is_contiguous() and v.get_device() == index
                    and ms.dtype is torch.float8_e8m0fnu and ms.numel() == blocks and ms.is_contiguous()
                    and ms.get_device() == index
                    and vs.dtype is torch.float8_e8m0fnu and vs.numel() == blocks and vs.is_contiguous()
                    and vs.get_device() == index
                    and (copy is None or (copy.dtype in _HALVES and copy.numel() == n and copy.is_contiguous()
                                          and copy.get_device() == index)))
            grad_type = _DTYPES[g.dtype]
        except (AttributeError, KeyError):
            fine = False
        if not fine:
            _refuse_byte_segment(i, p, g, (m, ms, v, vs), copy, device)
        if device is None:
            device = p.device
        written += (p, m, ms, v, vs)
        copied = address = 0
        if copy is not None:
            copied, address = _DTYPES[copy.dtype], copy.data_ptr()
            written.append(copy)
        _BYTE_SEGMENT.pack_into(buf, at, p.data_ptr(), g.data_ptr(), m.data_ptr(), ms.data_ptr(), v.data_ptr(),
                                vs.data_ptr(), address, n, grad_type, copied)
        at += _BYTE_SEGMENT.size
    hp = _AdamWByteHParams(lr, beta1, beta2, eps, weight_decay, int(step), int(bool(decoupled)),
                           int(bool(cautious_wd)))
    arr = (_AdamWByteSegment * len(segments)).from_buffer(buf)
    _call("ma_adamw_byte_step_multi", device, stream, arr, len(segments), ctypes.byref(hp), int(seed) & (2 ** 64 - 1))
    increment_version(written)
    if stream is not None:
        _record(stream, *written, *(s[1] for s in segments))


def _refuse_byte_segment(i, p, g, state, copy, device):
    """Raises what is wrong with a segment of adamw_byte_step_multi."""
    for name, t in (("param", p), ("grad", g)):
        _tensor(f"segment {i} {name}", t, device)
        device = t.device
    _require_f32_cuda(f"segment {i} param", p)
    n = p.numel()
    _type(f"segment {i} grad", g.dtype)
    if g.numel() != n or not g.is_contiguous():
        raise ValueError(f"segment {i} grad must be contiguous, of {n} values")
    for (name, dtype, block), t in zip(_ADAMW_BYTE_STATE, state):
        _tensor(f"segment {i} {name}", t, device)
        if t.dtype is not dtype or not t.is_contiguous() or t.numel() != -(-n // block):
            raise ValueError(f"segment {i} {name} must be contiguous {dtype} of {-(-n // block)} values "
                             f"(got {t.dtype}, {t.numel()})")
    if copy is not None:
        _tensor(f"segment {i} copy", copy, device)
    raise ValueError(f"segment {i} copy must be contiguous float16 or bfloat16 of {n} values")


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


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, post_weight, post_bias, gate, post_norm, scale, center, eps):
        ctx.set_materialize_grads(False)
        ctx.how = dict(post_norm=post_norm, scale=scale, center=center)
        out, y, stats = residual_norm_forward(x, residual, weight, bias, post_weight=post_weight, post_bias=post_bias,
                                              gate=gate, eps=eps, **ctx.how)
        ctx.save_for_backward(x, out, stats, weight, bias, post_weight, post_bias, gate)
        return out, y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dy):
        x, out, stats, *gains = ctx.saved_tensors
        if dout is None and dy is None:
            return (None,) * 11
        dout = dout if dout is None else _rowed(dout)
        dy = torch.zeros_like(out) if dy is None else _rowed(dy)
        weight, bias, post_weight, post_bias, gate = gains
        dx, dresidual, *grads = residual_norm_backward(dout, dy, x, out, stats, weight, bias, post_weight=post_weight,
                                                       post_bias=post_bias, gate=gate,
                                                       param_grads=ctx.needs_input_grad[2:7], **ctx.how)
        grads = [g if g is None else g.view(t.shape) for g, t in zip(grads, gains)]
        return dx, dresidual, *grads, None, None, None, None


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


class _HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, labels, copy):
        # (under autograd a weight of another type is the parameter that `copy` stands for)
        used = weight.detach().to(hidden.dtype) if copy is None else copy
        labels = labels.contiguous()
        loss, lse = head_loss_forward(hidden, used, labels)
        ctx.save_for_backward(hidden, used, labels, lse)
        ctx.dtype = weight.dtype
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        hidden, used, labels, lse = ctx.saved_tensors
        hidden_grad, weight_grad = ctx.needs_input_grad[:2]
        if not (hidden_grad or weight_grad):
            return None, None, None, None
        dweight = None
        if weight_grad and ctx.dtype != used.dtype:
            dweight = torch.empty(used.shape, dtype=ctx.dtype, device=used.device)
        dhidden, dweight = head_loss_backward(hidden, used, labels, lse, dloss.contiguous(), hidden_grad=hidden_grad,
                                              weight_grad=weight_grad, dweight=dweight)
        return dhidden, dweight, None, None


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


def residual_norm(x, residual, weight=None, bias=None, *, post_norm: bool = True, post_weight=None, post_bias=None,
                  gate=None, scale: float = 1.0, center: bool = True, eps: float = 1e-5):
    """(out, y): the residual stream behind a block with output x, and the next block's input (see
    residual_norm_forward); differentiable by x, the residual and all gains, biases and the gate."""
    return _ResidualNorm.apply(x, residual, weight, bias, post_weight, post_bias, gate, bool(post_norm), float(scale),
                               bool(center), float(eps))


def distill_loss(logits, teacher, ids, *, temperature: float = 1.0):
    """The distillation loss of each row (see distill_forward), differentiable by the logits;
    the teacher is constant."""
    return _DistillLoss.apply(logits, teacher, ids, float(temperature))


def head_loss(hidden, weight, labels, *, copy=None):
    """The softmax cross entropy of each label under the LM head's logits (see head_loss_forward),
    differentiable by the hidden states and the weight.  An fp32 weight under 16-bit hidden states
    is rounded to their type for the call, or `copy` is read in its place: the weight in that type,
    as a MuonAdamW group with 8-bit moments keeps it (`copies`).  The weight's gradient is fp32
    then."""
    if copy is not None and (copy.shape != weight.shape or copy.dtype != hidden.dtype):
        raise ValueError("copy must have the weight's shape and the hidden states' type")
    if weight.dtype not in (torch.float32, hidden.dtype):
        raise ValueError("weight must be float32 or have the hidden states' type")
    return _HeadLoss.apply(hidden, weight, labels, copy)
