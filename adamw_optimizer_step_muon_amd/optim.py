"""MuonAdamW: one optimizer over "muon" and "adamw" parameter groups.

"MuonAdamW vs DistMuonAdamW: Key Differences for Single and Multi-GPU Training in
nanochat": a single optimizer takes param_groups tagged ``"kind": "muon"`` or
``"kind": "adamw"`` with per-group hyperparameters; ``step()`` after ``backward()``;
the Muon kernel works on same-shape stacks (K, ...).  "Optimizers: AdamW, Muon and
the distributed optimizer", section "Muon: orthogonalising the update": Muon for
hidden 2-D matrices, AdamW for embeddings, the output layer and vectors.
"DMuon: Efficient Distributed Muon Training with Near-Adam Overhead", section 2.2
(batching): same-shape matrices are orthogonalised together.

Host bookkeeping only: each group is marshalled to the C ABI (one ma_muon_step over
all of a group's shape buckets, ma_adamw_step_multi over its AdamW tensors).

Muon parameters are bucketed by shape at construction: the K 2-D parameters of one
shape A x B become views into one contiguous (K, A, B) buffer (their values are copied
in, and ``p.data`` is re-pointed at the view, so the parameter objects the caller holds
see every update), and each parameter's momentum is a view into a (K, A, B) momentum
buffer.  A 3-D (K, A, B) parameter is a bucket of its own.  At each step the
gradients are gathered into one (K, A, B) buffer per bucket (one copy launch per
bucket; none when the gradients already are the buffer's views: the gather leaves
them so, and backward then accumulates into the buffer until ``zero_grad()`` drops
them), and a single ma_muon_step runs all buckets, so buckets that share a GEMM
configuration share its launches.  Parameters without a gradient are not stepped.
State is fp32 and zero-initialised: ``momentum_buffer`` (4 bytes per Muon parameter),
``exp_avg`` and ``exp_avg_sq`` (8 bytes per AdamW parameter).  An embedding table's gradient
can come as tokens and output gradients (``add_token_gradient``, which ``embedding(...,
optimizer=...)`` calls in its backward pass); its dense form is then never built.

An AdamW group's ``state_bits=8`` holds its moments in 8 bits instead (2 + 1/32 bytes per
parameter, see adamw_byte_step_multi): ``exp_avg``, ``exp_avg_sq`` and their blocks' scales, with
``seed`` for the roundings' random bits.  Its ``copies`` (one entry per parameter, None or a
contiguous fp16 or bf16 tensor of its size) receive the stepped parameters, for a forward pass
that reads 16-bit weights; what they hold before a parameter's first step is the caller's, but
load_state_dict writes them from the parameters (which are to be restored before it).  Token
gradients are built densely there.

A Muon group's ``ns_mode`` (0 by default) selects the Newton-Schulz route: 1 runs the
Gram-space iteration ("DMuon", section 2.2) on fp16 operands for the buckets whose long
side is at least 3.5x the other (MLP projections), the printed iteration elsewhere.
"""
from __future__ import annotations

from typing import Dict, List

from . import _lib

MUON_DEFAULTS = dict(lr=0.02, momentum=0.95, weight_decay=0.0, nesterov=True, ns_steps=5,
                     ns_coeffs=None, ns_eps=1e-7, cautious_wd=False, scale_mode=0, ns_mode=0)
ADAMW_DEFAULTS = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                      decoupled=True, cautious_wd=False, state_bits=32, seed=0, copies=None)


_F32_MAX = 3.4028234663852886e38


def _version(t):
    """t's version, None for the tensors of inference mode, which have none."""
    return None if t.is_inference() else t._version


def _stream_of(t):
    """(the current stream of t's device, whether a graph is being captured on it)."""
    import torch

    if not t.is_cuda:
        return None
    with torch.cuda.device(t.device):
        return torch.cuda.current_stream(), torch.cuda.is_current_stream_capturing()


def _order_behind(made_on, t) -> None:
    """The current stream waits for what a token gradient was made on, if that is another: a
    backward pass runs on its forward pass's stream, and torch orders its caller's stream
    behind the gradients that it sets itself.  Between a captured part and an eager one, or two
    captures, there is nothing to record: captures begin on an idle device, and replays are the
    caller's to order."""
    import torch

    if made_on is None:  # no GPU tensors: refused by the call that follows
        return
    here, capturing = _stream_of(t)
    stream, captured = made_on
    if stream == here or captured != capturing:
        return
    if captured:
        with torch.cuda.stream(stream):
            if not torch.cuda.is_current_stream_capturing():
                return
    here.wait_stream(stream)


class _Bucket:
    """K same-shape Muon parameters stored as one (K, A, B) buffer."""

    def __init__(self, params, stacked: bool):
        import torch

        self.params = params
        self.stacked = stacked  # one caller-provided (K, A, B) parameter
        if stacked:
            self.param = params[0].data
        else:
            self.param = torch.stack([p.data for p in params])
            for k, p in enumerate(params):
                p.data = self.param[k]
        self.grad = torch.zeros_like(self.param)
        self.momentum = torch.zeros_like(self.param)

    def momentum_view(self, k):
        return self.momentum if self.stacked else self.momentum[k]

    def live_stacks(self):
        """(param, grad, momentum) stacks for ma_muon_step: the whole bucket when every
        parameter has a gradient (gathered into the bucket's gradient buffer), one
        (1, A, B) slice per parameter that has one when only some do (a parameter
        without a gradient is not stepped; a matrix's result does not depend on the
        bucket it runs in), nothing when none does."""
        import torch

        grads = [p.grad for p in self.params]
        if all(g is None for g in grads):
            return []
        if self.stacked:
            if grads[0].data_ptr() != self.grad.data_ptr():
                self.grad.copy_(grads[0])
            return [(self.param, self.grad, self.momentum)]
        K = len(self.params)
        if any(g is None for g in grads):
            return [(self.param[k:k + 1], grads[k].reshape(1, *grads[k].shape).contiguous(),
                     self.momentum[k:k + 1]) for k in range(K) if grads[k] is not None]
        views = [self.grad[k] for k in range(K)]
        if not all(g.data_ptr() == v.data_ptr() for g, v in zip(grads, views)):
            torch.stack(grads, out=self.grad)
            # later backward passes accumulate straight into the buffer
            for p, v in zip(self.params, views):
                p.grad = v
        return [(self.param, self.grad, self.momentum)]

    @property
    def shape(self):
        return tuple(self.param.shape)


class MuonAdamW:
    def __init__(self, param_groups: List[Dict]):
        import torch

        self.param_groups = []
        self.state: Dict[int, Dict] = {}
        self._workspace = None
        self._buckets: Dict[int, List[_Bucket]] = {}
        # id(parameter) -> [(tokens, dout, scale, versions, stream)], see add_token_gradient
        self._token_grads: Dict[int, List] = {}
        for g in param_groups:
            kind = g.get("kind", "muon")
            if kind not in ("muon", "adamw"):
                raise ValueError(f"unknown group kind {kind!r}")
            defaults = MUON_DEFAULTS if kind == "muon" else ADAMW_DEFAULTS
            unknown = set(g) - set(defaults) - {"params", "kind"}
            if unknown:
                raise ValueError(f"unknown {kind} hyperparameters {sorted(unknown)}")
            group = dict(defaults)
            group.update(g)
            group["kind"] = kind
            group["params"] = list(g["params"])
            group["step"] = 0
            for p in group["params"]:
                if p.dtype != torch.float32 or not p.is_contiguous():
                    raise ValueError("parameters must be contiguous float32 tensors")
                if kind == "muon" and p.dim() not in (2, 3):
                    raise ValueError("Muon parameters are 2-D or (K, A, B) stacks")
            if len({id(p) for p in group["params"]}) != len(group["params"]):
                raise ValueError("a parameter appears twice in one group")
            if kind == "muon":
                buckets = self._bucket(group["params"])
                self._buckets[len(self.param_groups)] = buckets
                for b in buckets:
                    for k, p in enumerate(b.params):
                        self.state[id(p)] = {"momentum_buffer": b.momentum_view(k)}
            else:
                self._check_state_bits(group)
                for p in group["params"]:
                    self.state[id(p)] = self._byte_state(p) if group["state_bits"] == 8 else {
                        "exp_avg": torch.zeros_like(p), "exp_avg_sq": torch.zeros_like(p)}
            self.param_groups.append(group)

    @staticmethod
    def _check_state_bits(group) -> None:
        import torch

        if group["state_bits"] not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32 (got {group['state_bits']!r})")
        if group["copies"] is None:
            return
        if group["state_bits"] != 8:
            raise ValueError("copies are for groups with state_bits 8")
        group["copies"] = list(group["copies"])
        if len(group["copies"]) != len(group["params"]):
            raise ValueError("copies must have one entry per parameter")
        for p, c in zip(group["params"], group["copies"]):
            if c is not None and (c.dtype not in (torch.float16, torch.bfloat16) or c.device != p.device
                                  or c.numel() != p.numel() or not c.is_contiguous()):
                raise ValueError("copies must be contiguous float16 or bfloat16 tensors of their "
                                 "parameters' sizes")

    @staticmethod
    def _byte_state(p) -> Dict:
        from . import ops

        return dict(zip(("exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale"),
                        ops.adamw_byte_state(p)))

    @staticmethod
    def _bucket(params) -> List[_Bucket]:
        """Same-shape 2-D parameters into (K, A, B) buckets, in order of first appearance;
        each 3-D parameter a bucket of its own."""
        order, by_shape = [], {}
        for p in params:
            if p.dim() == 3:
                order.append(("stack", id(p), [p]))
                continue
            key = tuple(p.shape)
            if key not in by_shape:
                by_shape[key] = []
                order.append(("shape", key, by_shape[key]))
            by_shape[key].append(p)
        return [_Bucket(ps, kind == "stack") for kind, _, ps in order]

    def muon_buckets(self, group_index: int = None):
        """(K, A, B) of the Muon buckets (of one group, or of every Muon group)."""
        idx = [group_index] if group_index is not None else sorted(self._buckets)
        return [b.shape for i in idx for b in self._buckets.get(i, [])]

    def state_bytes_per_param(self, kind: str) -> float:
        n = b = 0
        for g in self.param_groups:
            if g["kind"] != kind:
                continue
            for p in g["params"]:
                n += p.numel()
                b += sum(t.numel() * t.element_size() for t in self.state[id(p)].values())
        return b / n if n else 0.0

    def _muon_workspace(self, shapes, device, ns_mode):
        import torch

        need = _lib.muon_workspace_bytes(shapes, ns_mode)
        if need and (self._workspace is None or self._workspace.numel() < need):
            self._workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return self._workspace

    def check_token_parameter(self, param) -> None:
        """Raises unless `param` can take token gradients (see add_token_gradient)."""
        if not any(q is param for g in self.param_groups if g["kind"] == "adamw"
                   for q in g["params"]):
            raise ValueError("token gradients are for parameters of an adamw group")
        if param.dim() != 2 or param.numel() == 0:
            raise ValueError("token gradients are for (rows, dim) parameters")

    def add_token_gradient(self, param, tokens, dout, scale: float = 1.0) -> None:
        """Adds to the gradient of an embedding table (a 2-D parameter of an "adamw" group)
        scale * dout[t] on row tokens[t] for every t, without building it: the next step()
        applies tokens and output gradients directly (adamw_step_embedding: no dense
        gradient is written or read).  Several additions, or one next to a dense
        ``param.grad`` or for a group with moments in 8 bits, are summed into ``param.grad`` at
        step() instead.  tokens (int32 or
        int64) and dout (tokens.shape + (dim,)) are kept, not copied, until zero_grad() and
        must not be modified before step(), which waits for the stream that is current here
        where its own is another.  What reads or changes ``param.grad`` between
        backward and step (clipping by a global norm, a loss scaler's unscaling) does not
        reach this gradient, and the ``scale`` that ``embedding`` hands over is that of its
        forward pass: a training loop that needs either leaves ``optimizer`` out there, or
        calls this once the factor is known, with a ``scale`` that holds it."""
        import torch

        self.check_token_parameter(param)
        if dout.shape != tokens.shape + (param.shape[1],):
            raise ValueError("dout must be tokens.shape + (dim,) of a (rows, dim) parameter")
        if tokens.dtype not in (torch.int32, torch.int64) or \
                dout.dtype not in (torch.float32, torch.float16, torch.bfloat16):
            raise ValueError("tokens must be int32 or int64, dout float32, float16 or bfloat16")
        if tokens.device != param.device or dout.device != param.device:
            raise ValueError("tokens and dout must be on the parameter's device")
        scale = float(scale)
        if not abs(scale) <= _F32_MAX:
            raise ValueError("scale must be finite in fp32")
        from . import ops

        ops._rows("dout", dout, anywhere=True)  # raises where they have no common stride
        self._token_grads.setdefault(id(param), []).append(
            (tokens, dout, scale, (_version(tokens), _version(dout)), _stream_of(param)))

    def _check_token_gradients(self) -> None:
        """Raises what step() would find wrong with a token gradient, before it changes
        anything."""
        if not self._token_grads:
            return
        for g in self.param_groups:
            for p in g["params"]:
                for tokens, dout, _, versions, _ in self._token_grads.get(id(p), ()):
                    if (_version(tokens), _version(dout)) != versions:
                        raise RuntimeError("the tokens or output gradients of a token gradient "
                                           "were modified before step()")
                    if p.grad is not None:
                        _lib._require_f32_cuda("the grad that token gradients add to", p.grad)

    def _take_token_gradient(self, p, direct: bool):
        """The token gradient to step p with directly, or None where p.grad holds it all."""
        added = self._token_grads.get(id(p))
        if not added:
            return None
        if direct and len(added) == 1 and p.grad is None:
            return added[0]
        from . import ops

        while added:  # what p.grad holds is no longer in the list
            tokens, dout, scale, _, made_on = added[0]
            _order_behind(made_on, p)
            ops.record_use(tokens, dout)
            if p.grad is None:
                p.grad = ops.embedding_backward(dout, tokens, p.shape[0], scale=scale)
            else:
                ops.embedding_backward(dout, tokens, p.shape[0], scale=scale, grad=p.grad,
                                       accumulate=True)
            del added[0]
        del self._token_grads[id(p)]
        return None

    def step(self) -> None:
        self._check_token_gradients()
        for gi, g in enumerate(self.param_groups):
            if g["kind"] == "adamw":
                by_token = [(p, t) for p in g["params"]
                            for t in [self._take_token_gradient(p, g["state_bits"] == 32)]
                            if t is not None]
                live = [p for p in g["params"] if p.grad is not None]
                if not live and not by_token:
                    continue
                b1, b2 = g["betas"]
                hp = dict(step=g["step"] + 1, lr=g["lr"], beta1=b1, beta2=b2, eps=g["eps"],
                          weight_decay=g["weight_decay"], decoupled=g["decoupled"],
                          cautious_wd=g["cautious_wd"])
                if g["state_bits"] == 8:
                    from . import ops

                    copies = g["copies"] or [None] * len(g["params"])
                    ops.adamw_byte_step_multi(
                        [(p.data, p.grad, *self.state[id(p)].values(), c)
                         for p, c in zip(g["params"], copies) if p.grad is not None],
                        seed=g["seed"], **hp)
                    g["step"] += 1
                    continue
                # the group's tensors in one fused pass (one launch per 48 tensors)
                segs = [(p.data, p.grad, self.state[id(p)]["exp_avg"],
                         self.state[id(p)]["exp_avg_sq"]) for p in live]
                _lib.adamw_step_multi(segs, **hp)
                for p, (tokens, dout, scale, _, made_on) in by_token:
                    from . import ops

                    _order_behind(made_on, p)
                    ops.adamw_step_embedding(p.data, tokens, dout, self.state[id(p)]["exp_avg"],
                                             self.state[id(p)]["exp_avg_sq"], scale=scale, **hp)
                    # perhaps another stream's memory, and dropped by zero_grad()
                    ops.record_use(tokens, dout)
                g["step"] += 1
                continue
            # Muon: every bucket with gradients in one call
            stacks = [st for b in self._buckets[gi] for st in b.live_stacks()]
            if not stacks:
                continue
            g["step"] += 1
            ws = self._muon_workspace([tuple(st[0].shape) for st in stacks], stacks[0][0].device,
                                      g["ns_mode"])
            _lib.muon_step(stacks, lr=g["lr"], momentum=g["momentum"],
                           weight_decay=g["weight_decay"], nesterov=g["nesterov"],
                           ns_steps=g["ns_steps"], ns_coeffs=g["ns_coeffs"], ns_eps=g["ns_eps"],
                           cautious_wd=g["cautious_wd"], scale_mode=g["scale_mode"],
                           ns_mode=g["ns_mode"], workspace=ws)

    def zero_grad(self, set_to_none: bool = True) -> None:
        self._token_grads.clear()
        for g in self.param_groups:
            for p in g["params"]:
                if p.grad is None:
                    continue
                if set_to_none:
                    p.grad = None
                else:
                    p.grad.zero_()

    def state_dict(self) -> Dict:
        groups, state = [], {}
        idx = 0
        for g in self.param_groups:
            ids = []
            for p in g["params"]:
                state[idx] = {k: v.clone() for k, v in self.state[id(p)].items()}
                ids.append(idx)
                idx += 1
            groups.append({k: v for k, v in g.items() if k not in ("params", "copies")} | {"params": ids})
        return {"state": state, "param_groups": groups}

    def load_state_dict(self, sd: Dict) -> None:
        import torch

        flat = [p for g in self.param_groups for p in g["params"]]
        for (idx, st) in sd["state"].items():
            # 8-bit moments mean nothing without their scales, and a cast would lose most values
            if ("exp_avg_scale" in st) != ("exp_avg_scale" in self.state[id(flat[int(idx)])]):
                raise ValueError("the state's moments have another number of bits (state_bits)")
        for (idx, st) in sd["state"].items():
            for k, v in st.items():
                self.state[id(flat[int(idx)])][k].copy_(v)
        for g, sg in zip(self.param_groups, sd["param_groups"]):
            g["step"] = sg["step"]
            # a forward pass before the next step reads what the parameters are now
            with torch.no_grad():
                for p, c in zip(g["params"], g.get("copies") or ()):
                    if c is not None:
                        c.copy_(p.view(c.shape))
