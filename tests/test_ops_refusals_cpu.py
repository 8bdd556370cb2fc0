"""What the training operators refuse, before anything is launched (no GPU needed: every
call below fails its checks on the host), and what the binding refuses."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")
from adamw_optimizer_step_muon_amd import _lib  # noqa: E402

INVALID, UNSUPPORTED, WORKSPACE = (_lib.MA_ERR_INVALID_ARG, _lib.MA_ERR_UNSUPPORTED,
                                   _lib.MA_ERR_WORKSPACE)
NAN = float("nan")
# far apart, never dereferenced
A, B, C, D, F, G = ((i + 1) << 40 for i in range(6))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmuonadamw.so not built")
    return _lib.load()


def _refused(lib, name, defaults, changes, status):
    args = dict(defaults)
    assert set(changes) <= set(args)
    args.update(changes)
    assert getattr(lib, name)(*args.values()) == status, (name, changes)
    assert lib.ma_last_error()


LOOKUP = dict(table=A, rows=100, dim=8, tokens=B, bits=64, n=10, scale=1.0, out=C, type=2, stride=8,
              stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(table=None), INVALID), (dict(tokens=None), INVALID), (dict(out=None), INVALID),
    (dict(table=A + 2), INVALID), (dict(tokens=B + 4), INVALID), (dict(out=C + 1), INVALID),
    (dict(rows=0), INVALID), (dict(dim=0), INVALID), (dict(n=-1), INVALID), (dict(bits=16), INVALID),
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(stride=7), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=float("inf")), INVALID), (dict(out=A + 64), INVALID),
    (dict(out=B), INVALID), (dict(rows=2 ** 31 - 1), UNSUPPORTED), (dict(dim=2 ** 20 + 1), UNSUPPORTED),
    (dict(n=2 ** 30 + 1), UNSUPPORTED), (dict(stride=2 ** 41), UNSUPPORTED),
])
def test_lookup(lib, changes, status):
    _refused(lib, "ma_embedding_forward", LOOKUP, changes, status)


GRAD = dict(tokens=A, bits=64, n=1000, dout=B, type=2, stride=8, scale=1.0, grad=C, rows=100, dim=8,
            accumulate=0, ws=D, size=1 << 20, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(tokens=None), INVALID), (dict(dout=None), INVALID), (dict(grad=None), INVALID),
    (dict(grad=C + 2), INVALID), (dict(dout=B + 1), INVALID), (dict(bits=8), INVALID),
    (dict(type=9), INVALID), (dict(n=-5), INVALID), (dict(stride=3), INVALID), (dict(scale=NAN), INVALID),
    (dict(dout=C), INVALID), (dict(tokens=C + 16), INVALID), (dict(ws=C), INVALID), (dict(ws=B), INVALID),
    (dict(tokens=D), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=D + 128), WORKSPACE),
    (dict(size=100), WORKSPACE), (dict(rows=0), INVALID), (dict(rows=1 << 33), UNSUPPORTED),
])
def test_table_gradient(lib, changes, status):
    _refused(lib, "ma_embedding_backward", GRAD, changes, status)
    need = ma.embedding_workspace_bytes(100, 8, 1000)
    assert 0 < need < 1 << 20
    assert lib.ma_embedding_backward(*{**GRAD, "size": need - 1}.values()) == WORKSPACE


def test_workspace_sizes(lib):
    assert ma.embedding_workspace_bytes(100, 8, 0) == ma.embedding_workspace_bytes(100, 8, 256) == 0
    assert ma.embedding_workspace_bytes(0, 8, 5) == ma.embedding_workspace_bytes(5, 8, -1) == 0
    # two copies of keys and places, two words a row, little else for few tokens
    assert 8 * 50000 <= ma.embedding_workspace_bytes(50000, 64, 257) < 8 * 50000 + (1 << 17)
    # the partial sums stay a small share of the output gradients
    n, dim = 65536, 2048
    assert ma.embedding_workspace_bytes(128000, dim, n) < 16 * n + 8 * 128000 + n * dim // 4
    assert ma.layer_norm_workspace_bytes(0, 64) == ma.layer_norm_workspace_bytes(5, 0) == 0
    assert ma.layer_norm_workspace_bytes(5, 64) > 0


def _hp(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, decoupled=1,
                cautious_wd=0)
    base.update(kw)
    return _lib._AdamWHParams(**base)


STEP = dict(param=A, m=B, v=C, rows=100, dim=8, tokens=D, bits=32, n=1000, dout=F, type=0, stride=8,
            scale=1.0, hp=None, ws=G, size=1 << 20, stream=None)


@pytest.mark.parametrize("changes,hp,status", [
    (dict(), dict(step=0), INVALID), (dict(), dict(lr=NAN), INVALID), (dict(), dict(beta1=1.0), INVALID),
    (dict(param=None), {}, INVALID), (dict(m=A), {}, INVALID), (dict(v=B + 400), {}, INVALID),
    (dict(dout=A + 32), {}, INVALID), (dict(tokens=C), {}, INVALID), (dict(ws=A), {}, INVALID),
    (dict(ws=None), {}, WORKSPACE), (dict(size=0), {}, WORKSPACE), (dict(bits=0), {}, INVALID),
    (dict(type=4), {}, INVALID), (dict(scale=NAN), {}, INVALID), (dict(param=A + 1), {}, INVALID),
])
def test_table_step(lib, changes, hp, status):
    _refused(lib, "ma_adamw_step_embedding", {**STEP, "hp": ctypes.byref(_hp(**hp))}, changes, status)
    assert lib.ma_adamw_step_embedding(*STEP.values()) == INVALID  # no hyperparameters


NORM = dict(x=A, type=2, xs=64, n=10, dim=64, w=B, b=C, eps=1e-5, y=D, ys=64, mean=F, rstd=G, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(x=A + 1), INVALID), (dict(w=B + 2), INVALID), (dict(xs=63), INVALID), (dict(ys=1), INVALID),
    (dict(type=7), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=NAN), INVALID), (dict(dim=0), INVALID),
    (dict(n=-1), INVALID), (dict(y=A), INVALID), (dict(y=A + 100), INVALID), (dict(mean=G), INVALID),
    (dict(rstd=B), INVALID), (dict(y=C), INVALID), (dict(dim=2 ** 20 + 1, xs=2 ** 21, ys=2 ** 21), UNSUPPORTED),
    (dict(n=1 << 22), UNSUPPORTED),
])
def test_norm(lib, changes, status):
    _refused(lib, "ma_layer_norm_forward", NORM, changes, status)


NORM_GRAD = dict(dy=A, dys=64, x=B, xs=64, type=2, n=10, dim=64, w=None, mean=C, rstd=C + 4096, dx=D,
                 dxs=64, dw=F, db=F + 4096, accumulate=0, ws=G, size=1 << 20, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(dx=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dys=8), INVALID), (dict(dxs=8), INVALID), (dict(type=5), INVALID),
    (dict(dx=A), INVALID), (dict(dx=B), INVALID), (dict(dw=F + 4096), INVALID), (dict(dw=A), INVALID),
    (dict(db=F + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=G + 4), WORKSPACE),
    (dict(size=8), WORKSPACE), (dict(ws=B), INVALID), (dict(n=-2), INVALID), (dict(dim=-2), INVALID),
])
def test_norm_gradient(lib, changes, status):
    _refused(lib, "ma_layer_norm_backward", NORM_GRAD, changes, status)


DISTILL = dict(z=A, type=2, stride=500, n=10, vocab=500, teacher=B, teacher_type=0, ids=C, bits=64, top=5,
               tau=1.0)


@pytest.mark.parametrize("changes,status", [
    (dict(z=None), INVALID), (dict(z=A + 1), INVALID), (dict(teacher=None), INVALID), (dict(ids=None), INVALID),
    (dict(ids=C + 4), INVALID), (dict(type=3), INVALID), (dict(teacher_type=3), INVALID), (dict(bits=31), INVALID),
    (dict(stride=499), INVALID), (dict(n=-1), INVALID), (dict(vocab=0), INVALID), (dict(top=-1), INVALID),
    (dict(top=1025), UNSUPPORTED), (dict(tau=0.0), INVALID), (dict(tau=-1.0), INVALID), (dict(tau=NAN), INVALID),
    (dict(tau=float("inf")), INVALID), (dict(tau=1e-9), UNSUPPORTED), (dict(tau=1e9), UNSUPPORTED),
    (dict(n=1 << 22), UNSUPPORTED), (dict(vocab=1 << 31, stride=1 << 31), UNSUPPORTED),
])
def test_distill(lib, changes, status):
    _refused(lib, "ma_distill_forward", {**DISTILL, "loss": D, "stats": F, "stream": None}, changes, status)
    _refused(lib, "ma_distill_backward", {**DISTILL, "stats": D, "w": F, "dz": G, "dzs": 500, "stream": None},
             changes, status)
    _refused(lib, "ma_distill_loss_grad", {**DISTILL, "w": D, "loss": F, "dz": G, "dzs": 500, "stream": None},
             changes, status)


@pytest.mark.parametrize("name,changes", [
    ("ma_distill_forward", dict(loss=None)), ("ma_distill_forward", dict(stats=None)),
    ("ma_distill_forward", dict(loss=A)), ("ma_distill_forward", dict(stats=D)),
    ("ma_distill_forward", dict(stats=C)),
    ("ma_distill_backward", dict(stats=None)), ("ma_distill_backward", dict(w=None)),
    ("ma_distill_backward", dict(dz=None)), ("ma_distill_backward", dict(dzs=20)),
    ("ma_distill_backward", dict(dz=A + 2)), ("ma_distill_backward", dict(dz=A, dzs=501)),
    ("ma_distill_backward", dict(dz=F)), ("ma_distill_backward", dict(dz=B)),
    ("ma_distill_loss_grad", dict(w=None)), ("ma_distill_loss_grad", dict(loss=None)),
    ("ma_distill_loss_grad", dict(loss=D)), ("ma_distill_loss_grad", dict(loss=A)),
    ("ma_distill_loss_grad", dict(dz=F)), ("ma_distill_loss_grad", dict(dz=C)),
    ("ma_distill_loss_grad", dict(dz=A + 4)),
])
def test_distill_outputs(lib, name, changes):
    tail = {"ma_distill_forward": dict(loss=D, stats=F), "ma_distill_backward": dict(stats=D, w=F, dz=G, dzs=500),
            "ma_distill_loss_grad": dict(w=D, loss=F, dz=G, dzs=500)}[name]
    _refused(lib, name, {**DISTILL, **tail, "stream": None}, changes, INVALID)


def test_nothing_to_do_is_not_an_error(lib):
    assert lib.ma_embedding_forward(*{**LOOKUP, "n": 0, "table": None}.values()) == 0
    assert lib.ma_embedding_backward(*{**GRAD, "n": 0, "accumulate": 1, "tokens": None, "dout": None,
                                       "ws": None, "size": 0}.values()) == 0
    assert lib.ma_layer_norm_forward(*{**NORM, "n": 0}.values()) == 0
    assert lib.ma_layer_norm_backward(*{**NORM_GRAD, "n": 0, "accumulate": 1, "ws": None, "size": 0}.values()) == 0
    d = {**DISTILL, "n": 0}
    assert lib.ma_distill_forward(*d.values(), D, F, None) == 0
    assert lib.ma_distill_backward(*d.values(), D, F, G, 500, None) == 0
    assert lib.ma_distill_loss_grad(*d.values(), D, F, G, 500, None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    f, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        ma.embedding_forward(f, i)
    with pytest.raises(ValueError, match="GPU"):
        ma.embedding_backward(f, i, 10)
    with pytest.raises(ValueError, match="accumulate"):
        ma.embedding_backward(f, i, 10, accumulate=True)
    with pytest.raises(ValueError, match="GPU"):
        ma.adamw_step_embedding(f, i, f, f, f, step=1, lr=1e-3)
    with pytest.raises(ValueError, match="GPU"):
        ma.layer_norm_forward(f)
    with pytest.raises(ValueError, match="GPU"):
        ma.layer_norm_backward(f, f, f[:, 0], f[:, 0])
    with pytest.raises(ValueError, match="GPU"):
        ma.distill_forward(f, f, i)
    with pytest.raises(TypeError):
        ma.layer_norm_forward([1.0])
    with pytest.raises(AttributeError):
        ma.no_such_operator  # noqa: B018


def test_token_gradients_are_checked_when_added():
    table, other = torch.zeros(10, 4), torch.zeros(3, 4)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [table]}])
    tokens = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="adamw group"):
        opt.add_token_gradient(other, tokens, torch.zeros(5, 4))
    with pytest.raises(ValueError, match="dout"):
        opt.add_token_gradient(table, tokens, torch.zeros(5, 3))
    with pytest.raises(ValueError, match="int32"):
        opt.add_token_gradient(table, tokens.float(), torch.zeros(5, 4))
    with pytest.raises(ValueError, match="float32"):
        opt.add_token_gradient(table, tokens, torch.zeros(5, 4).double())
    with pytest.raises(ValueError, match="adamw group"):
        ma.embedding(tokens, other, optimizer=opt)
    dout = torch.zeros(5, 4)
    opt.add_token_gradient(table, tokens, dout)
    dout.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        opt.step()
    opt.zero_grad()
    opt.step()  # nothing left to step


def test_token_gradients_that_a_step_would_refuse_are_refused_when_added():
    table, empty = torch.zeros(10, 4), torch.zeros(0, 4)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [table, empty]}])
    tokens, dout = torch.zeros(6, dtype=torch.int64), torch.zeros(6, 4)
    for bad in (dout[:1].expand(6, 4), torch.zeros(4, 6).t()):
        with pytest.raises(ValueError, match="rows"):
            opt.add_token_gradient(table, tokens, bad)
    with pytest.raises(ValueError, match="common stride"):
        opt.add_token_gradient(table, tokens.view(2, 3), torch.zeros(2, 4, 4)[:, :3])
    for scale in (NAN, float("inf"), 1e39):
        with pytest.raises(ValueError, match="scale"):
            opt.add_token_gradient(table, tokens, dout, scale)
    with pytest.raises(ValueError, match="parameters"):
        opt.add_token_gradient(empty, tokens, dout)
    opt.step()  # nothing was added
    assert opt.param_groups[0]["step"] == 0


def test_a_step_that_refuses_a_token_gradient_changes_nothing():
    first, table = torch.zeros(3), torch.zeros(10, 4)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [first]}, {"kind": "adamw", "params": [table]}])
    tokens, dout = torch.zeros(5, dtype=torch.int64), torch.zeros(5, 4)
    first.grad = torch.zeros(3)
    opt.add_token_gradient(table, tokens, dout)
    opt.add_token_gradient(table, tokens, dout.clone())
    dout.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        opt.step()
    assert table.grad is None and [g["step"] for g in opt.param_groups] == [0, 0]


def test_token_gradients_of_inference_mode():
    """Its tensors have no version to check."""
    table = torch.zeros(10, 4)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [table]}])
    with torch.inference_mode():
        tokens, dout = torch.zeros(5, dtype=torch.int64), torch.zeros(5, 4)
    opt.add_token_gradient(table, tokens, dout)
    with pytest.raises(ValueError, match="GPU"):  # and no complaint about versions
        opt.step()


def test_star_import_with_and_without_torch():
    """Without torch there are the names that need none; with it the operators too."""
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(_lib.__file__)))
    hide = ("import sys, importlib.util as u; find = u.find_spec; "
            "u.find_spec = lambda name, *a: None if name == 'torch' else find(name, *a); sys.modules['torch'] = None; ")
    check = "from adamw_optimizer_step_muon_amd import *; print('muon_step' in dir(), 'layer_norm' in dir())"
    for code, want in ((hide + check, "True False"), (check, "True True")):
        out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
        assert out.stdout.strip() == want, out.stderr


def test_binding_refuses_what_is_no_tensor():
    i = torch.zeros(4, dtype=torch.int64)
    for bad in (None, [1.0], 3):
        with pytest.raises(TypeError, match="dout"):
            ma.embedding_backward(bad, i, 10)


BYTE = dict(param=A, grad=B, exp_avg=C, exp_avg_scale=C + 4096, exp_avg_sq=D, exp_avg_sq_scale=D + 4096, copy=F, n=1000,
            grad_type=2, copy_type=2)


def _byte_hp(**kw):
    return _lib._AdamWByteHParams(**{**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, decoupled=1,
                                            cautious_wd=0), **kw})


def _byte_step(lib, *segments, n=None, hp={}, seed=0):
    arr = (_lib._AdamWByteSegment * len(segments))(*(_lib._AdamWByteSegment(*s.values()) for s in segments))
    return lib.ma_adamw_byte_step_multi(arr, len(segments) if n is None else n, ctypes.byref(_byte_hp(**hp)), seed, None)


@pytest.mark.parametrize("changes,status", [
    (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(exp_avg=None), INVALID),
    (dict(exp_avg_scale=None), INVALID), (dict(exp_avg_sq=None), INVALID), (dict(exp_avg_sq_scale=None), INVALID),
    (dict(param=A + 2), INVALID), (dict(grad=B + 1), INVALID), (dict(grad=B + 2, grad_type=0), INVALID),
    (dict(copy=F + 1), INVALID), (dict(grad_type=3), INVALID), (dict(grad_type=-1), INVALID), (dict(copy_type=0), INVALID),
    (dict(copy_type=3), INVALID), (dict(n=-1), INVALID), (dict(grad=A + 3998), INVALID), (dict(exp_avg=A), INVALID),
    (dict(exp_avg_scale=C + 999), INVALID), (dict(exp_avg_sq=C), INVALID), (dict(exp_avg_sq_scale=C + 4096 + 15), INVALID),
    (dict(copy=A), INVALID), (dict(copy=B), INVALID), (dict(n=1 << 37), UNSUPPORTED),
])
def test_byte_step(lib, changes, status):
    assert set(changes) <= set(BYTE)
    assert _byte_step(lib, {**BYTE, **changes}) == status and lib.ma_last_error()


def test_byte_step_lists(lib):
    other = {k: v + (1 << 30) if v is not None and k not in ("n", "grad_type", "copy_type") else v for k, v in BYTE.items()}
    assert _byte_step(lib, BYTE, dict(other, param=BYTE["copy"])) == INVALID
    assert _byte_step(lib, BYTE, dict(other, grad=BYTE["exp_avg"])) == INVALID
    assert _byte_step(lib, BYTE, n=-1) == INVALID
    assert _byte_step(lib, BYTE, hp=dict(step=0)) == INVALID
    assert _byte_step(lib, BYTE, hp=dict(lr=NAN)) == INVALID
    assert _byte_step(lib, BYTE, hp=dict(eps=1e300)) == INVALID  # no fp32 number
    assert _byte_step(lib, BYTE, hp=dict(beta2=1.0)) == INVALID
    assert lib.ma_adamw_byte_step_multi(None, 1, ctypes.byref(_byte_hp()), 0, None) == INVALID
    assert lib.ma_adamw_byte_step_multi(None, 0, ctypes.byref(_byte_hp()), 0, None) == 0
    assert lib.ma_adamw_byte_step_multi(None, 0, None, 0, None) == INVALID


def test_byte_state():
    p = torch.zeros(5, 13)
    m, ms, v, vs = ma.adamw_byte_state(p)
    assert m.shape == v.shape == p.shape and ms.shape == vs.shape == (2,)
    assert (m.dtype, ms.dtype, v.dtype) == (torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float8_e5m2)
    assert len({t.data_ptr() for t in (m, ms, v, vs)}) == 4
    assert torch.equal(ma.adamw_byte_values(m, ms), p)
    m.view(torch.uint8).fill_(torch.tensor(1.5).to(torch.float8_e4m3fn).view(torch.uint8).item())
    ms.view(torch.uint8)[1] = 129
    want = torch.full((65,), 1.5)
    want[64] = 6.0
    assert torch.equal(ma.adamw_byte_values(m, ms), want.view(5, 13))


def test_byte_group_refusals():
    p = torch.nn.Parameter(torch.zeros(4, 3))
    for bad in (dict(state_bits=16), dict(copies=[None]), dict(state_bits=8, copies=[]),
                dict(state_bits=8, copies=[torch.zeros(12)]), dict(state_bits=8, copies=[torch.zeros(11, dtype=torch.bfloat16)])):
        with pytest.raises(ValueError):
            ma.MuonAdamW([{"kind": "adamw", "params": [p], **bad}])
    with pytest.raises(ValueError, match="GPU"):
        ma.adamw_byte_step_multi([(p.data, p.data, *ma.adamw_byte_state(p))], step=1, lr=1e-3)
    with pytest.raises(TypeError):
        ma.adamw_byte_step_multi([(None, p.data, *ma.adamw_byte_state(p))], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="6 or 7"):
        ma.adamw_byte_step_multi([(p.data, p.data)], step=1, lr=1e-3)
    ma.adamw_byte_step_multi([], step=1, lr=1e-3)


HEAD = dict(h=A, type=2, hs=64, n=10, dim=64, w=B, ws=64, vocab=1000, labels=C, bits=64)
HEAD_FORWARD = dict(HEAD, loss=D, lse=D + 4096, space=F, size=1 << 40, stream=None)
HEAD_GRADS = dict(dh=G, dhs=64, dw=G + (1 << 30), dwt=0, dws=64, add=0, space=F, size=1 << 38, stream=None)
HEAD_BACKWARD = dict(HEAD, lse=D, rw=D + 4096, **HEAD_GRADS)
HEAD_GRAD = dict(HEAD, rw=D, loss=D + 4096, **HEAD_GRADS)
HEAD_BAD = [
    (dict(h=None), INVALID), (dict(w=None), INVALID), (dict(labels=None), INVALID), (dict(h=A + 1), INVALID),
    (dict(w=B + 1), INVALID), (dict(labels=C + 4), INVALID), (dict(type=3), INVALID), (dict(bits=16), INVALID),
    (dict(hs=63), INVALID), (dict(ws=8), INVALID), (dict(n=-1), INVALID), (dict(dim=0), INVALID), (dict(vocab=0), INVALID),
    (dict(space=None), WORKSPACE), (dict(space=F + 64), WORKSPACE), (dict(size=1000), WORKSPACE), (dict(space=A), INVALID),
    (dict(space=B), INVALID), (dict(n=1 << 22), UNSUPPORTED), (dict(dim=2 ** 20 + 1, hs=1 << 21, ws=1 << 21), UNSUPPORTED),
    (dict(vocab=2 ** 30 + 1), UNSUPPORTED), (dict(hs=1 << 41), UNSUPPORTED), (dict(n=1 << 21, vocab=1 << 29), UNSUPPORTED),
]


@pytest.mark.parametrize("changes,status", HEAD_BAD + [
    (dict(loss=None), INVALID), (dict(lse=None), INVALID), (dict(loss=D + 1), INVALID), (dict(loss=D + 4096), INVALID),
    (dict(lse=A + 8), INVALID), (dict(loss=C), INVALID), (dict(loss=B), INVALID)])
def test_head_forward(lib, changes, status):
    _refused(lib, "ma_head_loss_forward", HEAD_FORWARD, changes, status)


HEAD_BAD_GRADS = HEAD_BAD + [
    (dict(rw=None), INVALID), (dict(dwt=1), INVALID), (dict(dwt=2, add=1), INVALID), (dict(dhs=10), INVALID),
    (dict(dws=10), INVALID), (dict(dh=A), INVALID), (dict(dw=B), INVALID), (dict(dh=G + (1 << 30)), INVALID),
    (dict(dw=G + (1 << 30) + 2), INVALID), (dict(dh=G + 1), INVALID), (dict(dh=C), INVALID), (dict(dw=F + 256), INVALID)]


@pytest.mark.parametrize("changes,status", HEAD_BAD_GRADS + [(dict(lse=None), INVALID), (dict(dh=D), INVALID)])
def test_head_backward(lib, changes, status):
    _refused(lib, "ma_head_loss_backward", HEAD_BACKWARD, changes, status)


@pytest.mark.parametrize("changes,status", HEAD_BAD_GRADS + [(dict(loss=None), INVALID), (dict(loss=D), INVALID)])
def test_head_grad(lib, changes, status):
    _refused(lib, "ma_head_loss_grad", HEAD_GRAD, changes, status)


def test_head_workspace(lib):
    size = lambda n, dim, vocab, at=256, stride=None, grads=1, type=2: lib.ma_head_loss_workspace_bytes(  # noqa: E731
        type, n, dim, vocab, at, dim if stride is None else stride, grads)
    assert size(0, 64, 10) == size(5, 0, 10) == size(5, 64, 0) == size(5, 64, 10, type=3) == 0
    # a copy of the head only where its rows are not aligned
    for bad in (dict(at=258), dict(stride=68), dict(stride=1 << 23)):
        assert size(5, 64, 50000, **bad) - size(5, 64, 50000) == 50000 * 64 * 2
    assert size(5, 60, 50000, grads=0) - size(5, 64, 50000, grads=0) == 50000 * 64 * 2
    assert size(5, 60, 50000, at=4, type=0) == size(5, 60, 50000, type=0)
    # the logits of 8192 rows would take 2 GiB in 16 bits
    assert size(8192, 2048, 128000) < (512 << 20) + 8192 * 2048 * 2 * 8 + (1 << 20)
    assert size(8192, 2048, 128000, grads=0) < 100 << 20
    need = size(10, 64, 1000)
    assert lib.ma_head_loss_grad(*{**HEAD_GRAD, "size": need - 1}.values()) == WORKSPACE


def test_head_binding_refusals():
    h, w = torch.zeros(4, 8), torch.zeros(10, 8)
    with pytest.raises(ValueError, match="GPU"):
        ma.head_loss_forward(h, w, torch.zeros(4, dtype=torch.long))
    with pytest.raises(TypeError):
        ma.head_loss_forward(None, w, torch.zeros(4, dtype=torch.long))
    with pytest.raises(ValueError, match="copy"):
        ma.head_loss(h, w, torch.zeros(4, dtype=torch.long), copy=w.half())
    with pytest.raises(ValueError, match="float32"):
        ma.head_loss(h, w.half(), torch.zeros(4, dtype=torch.long))


RES_PARAMS = dict(post_weight=C, post_bias=C + 4096, gate=C + 8192, weight=C + 12288, bias=C + 16384, scale=0.5, eps=1e-5,
                  post_norm=1, center=1)
RES = dict(x=A, xs=64, res=B, rs=64, type=2, n=10, dim=64, params=None, out=D, outs=64, y=F, ys=64, stats=G, stream=None)


@pytest.mark.parametrize("changes,params,status", [
    (dict(x=None), {}, INVALID), (dict(res=None), {}, INVALID), (dict(out=None), {}, INVALID), (dict(y=None), {}, INVALID),
    (dict(stats=None), {}, INVALID), (dict(x=A + 1), {}, INVALID), (dict(stats=G + 2), {}, INVALID), (dict(type=5), {}, INVALID),
    (dict(xs=3), {}, INVALID), (dict(rs=63), {}, INVALID), (dict(outs=0), {}, INVALID), (dict(ys=1), {}, INVALID),
    (dict(n=-1), {}, INVALID), (dict(dim=0), {}, INVALID), (dict(out=A), {}, INVALID), (dict(out=B + 16), {}, INVALID),
    (dict(out=B, outs=65), {}, INVALID), (dict(y=B), {}, INVALID), (dict(y=D), {}, INVALID), (dict(stats=C), {}, INVALID),
    (dict(n=1 << 22), {}, UNSUPPORTED), (dict(dim=1 << 21), {}, UNSUPPORTED),
    ({}, dict(scale=NAN), INVALID), ({}, dict(eps=-1.0), INVALID), ({}, dict(eps=NAN), INVALID), ({}, dict(weight=C + 1), INVALID),
    ({}, dict(post_norm=0), INVALID), ({}, dict(post_norm=0, post_weight=None), INVALID), ({}, dict(gate=D), INVALID),
])
def test_residual_norm(lib, changes, params, status):
    p = _lib._ResidualNormParams(*{**RES_PARAMS, **params}.values())
    _refused(lib, "ma_residual_norm_forward", dict(RES, params=ctypes.byref(p)), changes, status)
    assert lib.ma_residual_norm_forward(*RES.values()) == INVALID  # no parameters


RES_GRAD = dict(dout=A, dos=64, dy=A + 4096, dys=64, x=B, xs=64, out=B + 4096, outs=64, stats=G, type=2, n=10, dim=64,
                params=None, grads=None, dx=D, dxs=64, dres=D + 4096, dress=64, ws=F, size=1 << 30, stream=None)
RES_GRADS = dict(dpost_weight=G + 4096, dpost_bias=G + 8192, dgate=G + 12288, dweight=G + 16384, dbias=G + 20480)


@pytest.mark.parametrize("changes,params,grads,status", [
    (dict(dy=None), {}, {}, INVALID), (dict(x=None), {}, {}, INVALID), (dict(out=None), {}, {}, INVALID),
    (dict(stats=None), {}, {}, INVALID), (dict(dx=None), {}, {}, INVALID), (dict(dres=None), {}, {}, INVALID),
    (dict(dos=1), {}, {}, INVALID), (dict(dys=1), {}, {}, INVALID), (dict(dxs=1), {}, {}, INVALID), (dict(dx=A), {}, {}, INVALID),
    (dict(dres=A + 4096), {}, {}, INVALID), (dict(dx=D + 4096), {}, {}, INVALID), (dict(ws=None), {}, {}, WORKSPACE),
    (dict(ws=F + 16), {}, {}, WORKSPACE), (dict(size=100), {}, {}, WORKSPACE), (dict(ws=B), {}, {}, INVALID),
    ({}, dict(post_norm=0, post_weight=None, post_bias=None), {}, INVALID), ({}, {}, dict(dgate=G + 4096), INVALID),
    ({}, {}, dict(dweight=G + 1), INVALID), ({}, {}, dict(dbias=C), INVALID), (dict(type=4), {}, {}, INVALID),
])
def test_residual_norm_gradient(lib, changes, params, grads, status):
    p = _lib._ResidualNormParams(*{**RES_PARAMS, **params}.values())
    g = _lib._ResidualNormGrads(*{**RES_GRADS, **grads}.values())
    args = dict(RES_GRAD, params=ctypes.byref(p), grads=ctypes.byref(g))
    _refused(lib, "ma_residual_norm_backward", args, changes, status)
    assert lib.ma_residual_norm_backward(*{**args, "grads": None}.values()) == INVALID
    assert ma.residual_norm_workspace_bytes(0, 64) == 0 < ma.residual_norm_workspace_bytes(5, 64)


def test_residual_norm_binding_refusals():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ma.residual_norm_forward(x, x)
    with pytest.raises(TypeError):
        ma.residual_norm_forward(None, x)


def test_byte_segment_layout():
    from adamw_optimizer_step_muon_amd import ops

    assert ops._BYTE_SEGMENT.size == ctypes.sizeof(_lib._AdamWByteSegment)
    raw = bytearray(ops._BYTE_SEGMENT.pack(1, 2, 3, 4, 5, 6, 7, -8, 1, 2))
    seg = _lib._AdamWByteSegment.from_buffer(raw)
    assert [getattr(seg, f) for f, _ in seg._fields_] == [1, 2, 3, 4, 5, 6, 7, -8, 1, 2]


def test_byte_segment_refusals():
    """Each tensor of a segment that is not as it has to be is named (on the CPU: none gets further
    than its device, so the checks are called with one)."""
    from adamw_optimizer_step_muon_amd import ops

    p = torch.zeros(70)
    for bad in (p.half(), torch.zeros(140)[::2], None):
        with pytest.raises((ValueError, TypeError), match="segment 3 param"):
            ops._refuse_byte_segment(3, bad, p, ma.adamw_byte_state(p), None, None)
