"""The norms around a block against the fp64 reference.

Bounds (e = 2^-24, u the type's half step, k = (D / 64 + 16) e the relative error of a row's sum, as
for layer norm):
  first norm: mean off by dm <= k mean|x| (0 without a mean), variance by a relative k + 8 e and dm^2,
    rstd by half of that and 3 e; the branch, whose factor scale gate w1 has three roundings, by
    |factor| (h (drstd + 7 e) + dm rstd) + 4 e |scale gate b1|; out by that and 2 e of its terms
  second norm: its input is off by eo; mean by mean eo + k mean|out|, a deviation by their sum f, the
    variance by 2 mean(|c| f) + mean f^2 + (k + 8 e) variance; rstd and y as above
Backward, from given statistics: h off by 2 e, the two means by (k + 6 e) of their terms' magnitudes;
d by ed = rstd (.. ) + 2 e |dout| + e |d|, which enters dx, its means and the column sums once, each with
its own sums' errors; a column sum over N rows by (N + 8) e of its terms' magnitudes.
"""
import numpy as np
import pytest

from oracle import training

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
E = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
SIZES = [(1, 1), (3, 2), (5, 33), (64, 64), (257, 100), (77, 200), (19, 768), (7, 1279), (6, 2048), (5, 2051),
         (3, 4096), (4, 8192), (3, 8195), (2, 16384), (2, 16391), (2, 40000)]
MODES = [dict(), dict(center=False), dict(post_norm=False), dict(post_norm=False, center=False)]
GAINS = ["all", "weights", "gate", "none"]


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _strided(x, extra, offset):
    n, d = x.shape
    buf = torch.full((n, d + extra), float("nan"), dtype=x.dtype, device=DEV)
    view = buf[:, offset:offset + d]
    view.copy_(x)
    return view


def _inputs(n, dim, dtype, seed, mode, gains):
    rng = np.random.default_rng(seed)
    rows = [torch.from_numpy(rng.standard_normal((n, dim)) * s + o).to(dtype).to(DEV)
            for s, o in ((2, 0.5), (3, -0.25), (1, 0), (1, 0))]
    vec = {k: torch.from_numpy((rng.standard_normal(dim)).astype(np.float32)).to(DEV)
           for k in ("weight", "bias", "post_weight", "post_bias", "gate")}
    keep = {"all": set(vec), "weights": {"weight", "post_weight"}, "gate": {"gate"}, "none": set()}[gains]
    if not mode.get("post_norm", True):
        keep -= {"post_weight", "post_bias"}
    return rows, {k: v if k in keep else None for k, v in vec.items()}


def _abs(t):
    return 1.0 if t is None else np.abs(_np(t))


def _norm_errors(x, f, mean, rstd, k):
    """Errors of a norm's mean and rstd (relative) for an input x off by f."""
    c = np.abs(x - mean[:, None])
    dm = np.where(mean == 0, 0.0, f.mean(1) + k * np.abs(x).mean(1))
    g = f + dm[:, None]
    var = (c ** 2).mean(1)
    dvar = 2 * (c * f).mean(1) + (g ** 2).mean(1) + (k + 8 * E) * var
    return c, dm, 0.55 * dvar * rstd ** 2 + 3 * E


@pytest.mark.parametrize("n,dim", SIZES + [(1500, 48)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("gains", GAINS)
def test_forward(n, dim, dtype, mode, gains):
    (x, res, _, _), vec = _inputs(n, dim, dtype, n + dim, mode, gains)
    scale, eps = 0.75, 1e-5
    kw = dict(vec, scale=scale, eps=eps, **mode)
    out, y, stats = ma.residual_norm_forward(x, res, **kw)
    eps64 = float(np.float32(eps))
    ro, ry, rs = training.residual_norm(_np(x), _np(res), **{k: _np(v) for k, v in vec.items()}, scale=scale, eps=eps64, **mode)
    X, R, k = _np(x), _np(res), (dim / 64 + 16) * E
    gate = scale * _abs(vec["gate"])
    A, B = gate * _abs(vec["post_weight"]), gate * (0.0 if vec["post_bias"] is None else _abs(vec["post_bias"]))
    if mode.get("post_norm", True):
        c, dm, dr = _norm_errors(X, np.zeros_like(X), rs[0], rs[1], k)
        h, r = c * rs[1][:, None], rs[1][:, None]
        assert (np.abs(_np(stats[0]) - rs[0]) <= dm + E * np.abs(rs[0])).all()
        assert (np.abs(_np(stats[1]) - rs[1]) <= rs[1] * dr).all()
    else:
        h, dm, dr, r = np.abs(X), np.zeros(n), np.zeros(n), 1.0
        assert not stats[:2].any()
    eo = A * (h * (dr[:, None] + 7 * E) + dm[:, None] * r * 1.01) + 4 * E * B + 2 * E * (np.abs(R) + A * h + B)
    u = torch.finfo(dtype).eps / 2
    assert (np.abs(_np(out) - ro) <= eo * 1.01 + u * (np.abs(ro) + eo) + TINY[dtype]).all()
    c, dm, dr = _norm_errors(ro, eo, rs[2], rs[3], k)
    assert (np.abs(_np(stats[2]) - rs[2]) <= (dm + 2 * E * np.abs(rs[2])) * 1.01).all()
    assert (np.abs(_np(stats[3]) - rs[3]) <= rs[3] * dr * 1.01).all()
    W, b = _abs(vec["weight"]), 0.0 if vec["bias"] is None else _abs(vec["bias"])
    r = rs[3][:, None]
    bound = W * r * (c * (dr[:, None] + 3 * E) + (eo + dm[:, None]) * 1.01) + 3 * E * (c * r * W + b)
    bound = bound * 1.01 + u * (np.abs(ry) + bound) + TINY[dtype]
    assert (np.abs(_np(y) - ry) <= bound).all()
    # strides, alignment, and the residual stepped in place
    again = ma.residual_norm_forward(_strided(x, dim % 3, dim % 3 // 2), _strided(res, 5, 3), **kw)
    assert all(torch.equal(s, t) for s, t in zip((out, y, stats), again))
    place = _strided(res, 3, 1)
    again = ma.residual_norm_forward(x, place, out=place, **kw)
    assert again[0] is place and all(torch.equal(s, t) for s, t in zip((out, y, stats), again))


@pytest.mark.parametrize("n,dim", SIZES + [(2000, 48), (1031, 520)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("gains", GAINS)
def test_backward(n, dim, dtype, mode, gains):
    (x, res, dy, dout), vec = _inputs(n, dim, dtype, 7 * n + dim, mode, gains)
    scale = -1.25
    out, _, stats = ma.residual_norm_forward(x, res, **vec, scale=scale, **mode)
    kw = dict(vec, scale=scale, **mode)
    got = ma.residual_norm_backward(dout, dy, x, out, stats, **kw)
    X, O, DY, DO, S = _np(x), _np(out), _np(dy), _np(dout), _np(stats)
    gains64 = {a: _np(vec[a]) for a in ("weight", "post_weight", "post_bias", "gate")}
    ref = training.residual_norm_grad(DO, DY, X, O, S, **gains64, scale=scale, **mode)
    post, center = mode.get("post_norm", True), mode.get("center", True)
    k, u = (dim / 64 + 16) * E, torch.finfo(dtype).eps / 2
    rd = ref[1]
    h2, r2 = np.abs(O - S[2][:, None]) * S[3][:, None], S[3][:, None]
    u2 = np.abs(DY) * _abs(vec["weight"])
    s1, s2 = u2.mean(1, keepdims=True) * center, (u2 * h2).mean(1, keepdims=True)
    ed = r2 * (s1 * (k + 6 * E) + h2 * s2 * (k + 12 * E) + 6 * E * (u2 + s1 + h2 * s2)) + 2 * E * np.abs(DO) + E * np.abs(rd)
    assert (np.abs(_np(got[1]) - rd) <= ed * 1.01 + u * (np.abs(rd) + ed) + TINY[dtype]).all()
    gate = abs(scale) * _abs(vec["gate"])
    A = gate * _abs(vec["post_weight"])
    eu = A * (ed + 4 * E * np.abs(rd))
    u1, h1 = A * np.abs(rd), np.abs(X)
    if post:
        r1 = S[1][:, None]
        h1 = np.abs(X - S[0][:, None]) * r1
        n1, n2 = u1.mean(1, keepdims=True) * center, (u1 * h1).mean(1, keepdims=True)
        en1 = (eu.mean(1, keepdims=True) + (k + 4 * E) * n1) * center
        en2 = (eu * h1).mean(1, keepdims=True) + (k + 8 * E) * n2
        eu = r1 * (eu + en1 + h1 * en2 + 8 * E * (u1 + n1 + h1 * n2))
    assert (np.abs(_np(got[0]) - ref[0]) <= eu * 1.01 + u * (np.abs(ref[0]) + eu) + TINY[dtype]).all()
    eS = (ed * h1).sum(0) + (n + 8) * E * (np.abs(rd) * h1).sum(0)
    eR = ed.sum(0) + (n + 8) * E * np.abs(rd).sum(0)
    SS, RR = (np.abs(rd) * h1).sum(0), np.abs(rd).sum(0)
    pb = 0.0 if vec["post_bias"] is None else _abs(vec["post_bias"])
    bounds = [(n + 8) * E * (np.abs(DY) * h2).sum(0), (n + 8) * E * np.abs(DY).sum(0), gate * (eS + 4 * E * SS),
              gate * (eR + 4 * E * RR), abs(scale) * (_abs(vec["post_weight"]) * (eS + 4 * E * SS) + pb * (eR + 4 * E * RR))]
    for name, g, r, b in zip(("weight", "bias", "post_weight", "post_bias", "gate"), got[2:], ref[2:], bounds):
        assert (g is None) == (vec[name] is None)
        if g is not None:
            assert (np.abs(_np(g) - r) <= b * 1.01).all(), name
    again = ma.residual_norm_backward(_strided(dout, 3, 2), _strided(dy, 1, 0), _strided(x, 2, 1), _strided(out, 4, 4), stats, **kw)
    assert all((s is None and t is None) or torch.equal(s, t) for s, t in zip(got, again))
    alone = ma.residual_norm_backward(dout, dy, x, out, stats, param_grads=False, **kw)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1]) and alone[2:] == (None,) * 5
    none = ma.residual_norm_backward(None, dy, x, out, stats, **kw)
    zero = ma.residual_norm_backward(torch.zeros_like(dy), dy, x, out, stats, **kw)
    assert all((s is None and t is None) or torch.equal(s, t) for s, t in zip(none, zero))


def test_no_rows():
    (x, res, dy, dout), vec = _inputs(1, 40, torch.bfloat16, 1, {}, "all")
    x, res, dy, dout = (t[:0] for t in (x, res, dy, dout))
    out, y, stats = ma.residual_norm_forward(x, res, **vec)
    assert out.shape == y.shape == (0, 40) and stats.shape == (4, 0)
    got = ma.residual_norm_backward(dout, dy, x, out, stats, **vec)
    assert all(not t.any() for t in got[2:])


@pytest.mark.parametrize("dim", [96, 1000, 9000, 20000])
def test_not_a_number_stays_in_its_row(dim):
    (x, res, dy, dout), vec = _inputs(9, dim, torch.bfloat16, 2, {}, "all")
    want = ma.residual_norm_forward(x, res, **vec)
    back = ma.residual_norm_backward(dout, dy, x, want[0], want[2], **vec)
    x2, res2 = x.clone(), res.clone()
    x2[3, 7], res2[8, 1] = float("nan"), float("inf")
    got = ma.residual_norm_forward(x2, res2, **vec)
    on = torch.ones(9, dtype=torch.bool, device=DEV)
    on[[3, 8]] = False
    assert all(torch.equal(a[on], b[on]) for a, b in zip(got[:2], want[:2])) and torch.equal(got[2][:, on], want[2][:, on])
    assert torch.isnan(got[1][~on]).all()
    got = ma.residual_norm_backward(dout, dy, x2, got[0], got[2], **vec)
    assert torch.equal(got[0][on], back[0][on]) and torch.equal(got[1][on], back[1][on])


@pytest.mark.parametrize("mode", MODES)
def test_autograd_by_differences(mode):
    (x, res, w1, w2), vec = _inputs(4, 12, torch.float32, 3, mode, "all")
    leaves = [t.clone().requires_grad_(True) for t in (x, res)]
    params = {k: None if v is None else torch.nn.Parameter(v.view(3, 4).clone()) for k, v in vec.items()}
    out, y = ma.residual_norm(leaves[0].view(2, 2, 12), leaves[1].view(2, 2, 12), **params, scale=0.5, **mode)
    ((out * w1.view_as(out)).sum() + (y * w2.view_as(y)).sum()).backward()

    def total(values):
        o, t, _ = training.residual_norm(values["x"], values["residual"], **{k: v if v is None else v.reshape(-1)
                                         for k, v in values.items() if k not in ("x", "residual")}, scale=0.5,
                                         eps=float(np.float32(1e-5)), **mode)
        return (o * _np(w1)).sum() + (t * _np(w2)).sum()

    values = {"x": _np(x), "residual": _np(res), **{k: _np(v) for k, v in vec.items()}}
    grads = {"x": leaves[0].grad, "residual": leaves[1].grad, **{k: None if p is None else p.grad for k, p in params.items()}}
    for name, v in values.items():
        if v is None:
            continue
        assert grads[name].shape == (params[name].shape if name in params else x.shape)
        g = _np(grads[name]).reshape(-1)
        for i in range(0, v.size, 5):
            at = []
            for sign in (1, -1):
                moved = v.copy()
                moved.reshape(-1)[i] += sign * 1e-5
                at.append(total({**values, name: moved}))
            assert abs((at[0] - at[1]) / 2e-5 - g[i]) < 2e-4 * max(1.0, abs(g[i])), (name, i)


def test_autograd_with_one_output_used():
    (x, res, w, _), vec = _inputs(5, 64, torch.bfloat16, 4, {}, "all")
    for use in (0, 1):
        a, b = x.clone().requires_grad_(True), res.clone().requires_grad_(True)
        outs = ma.residual_norm(a, b, **vec)
        (outs[use] * w).sum().backward()
        out, _, stats = ma.residual_norm_forward(x, res, **vec)
        dx, dr, *_ = ma.residual_norm_backward(w if use == 0 else None, torch.zeros_like(w) if use == 0 else w, x, out, stats, **vec)
        assert torch.equal(a.grad, dx) and torch.equal(b.grad, dr)
    # a sum's gradient is an expanded scalar
    a = x.clone().requires_grad_(True)
    out, y = ma.residual_norm(a, res, **vec)
    (out.sum() + y.sum()).backward()
    assert a.grad is not None


@pytest.mark.parametrize("dtype", TYPES)
def test_stream_and_graph(dtype):
    (x, res, dy, dout), vec = _inputs(300, 136, dtype, 5, {}, "all")
    run = lambda a, **kw: (lambda f: f + ma.residual_norm_backward(dout, dy, a, f[0], f[2], **vec, **kw))(  # noqa: E731
        ma.residual_norm_forward(a, res, **vec, **kw))
    want = run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(static)
    for scale in (1.0, 0.25, 1.0):
        static.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = run(x * scale)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [200, 9000, 20000])
def test_rows_far_apart(dtype, dim):
    """Offsets pass 32 bits, and what lies between the rows stays."""
    n, stride = 20, (1 << 27) + 13
    (x, res, dy, dout), vec = _inputs(n, dim, dtype, 7, {}, "all")
    want = ma.residual_norm_forward(x, res, **vec)
    back = ma.residual_norm_backward(dout, dy, x, want[0], want[2], **vec)
    wide = torch.empty(n * stride, dtype=dtype, device=DEV).as_strided((n, dim + 9), (stride, 1))
    wide.fill_(5.0)
    out = wide[:, :dim]
    far = [torch.empty(n * stride, dtype=dtype, device=DEV).as_strided((n, dim), (stride, 1)) for _ in range(4)]
    for a, t in zip(far, (x, res, dy, dout)):
        a.copy_(t)
    got = ma.residual_norm_forward(far[0], far[1], out=out, **vec)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (wide[:, dim:] == 5).all()
    got = ma.residual_norm_backward(far[3], far[2], far[0], out, got[2], **vec)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    # the residual in place
    ma.residual_norm_forward(far[0], far[1], out=far[1], **vec)
    assert torch.equal(far[1], want[0]) and torch.equal(far[0], x)


def test_plain_norm_matches_layer_norm():
    """With a branch of nothing, y is the layer norm of the residual."""
    (x, res, _, _), vec = _inputs(50, 520, torch.float32, 6, {}, "weights")
    out, y, stats = ma.residual_norm_forward(x, res, vec["weight"], post_norm=False, scale=0.0)
    ly, mean, rstd = ma.layer_norm_forward(res, vec["weight"])
    assert torch.equal(out, res) and torch.equal(y, ly) and torch.equal(stats[2], mean) and torch.equal(stats[3], rstd)
