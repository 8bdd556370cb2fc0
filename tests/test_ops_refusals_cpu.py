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
