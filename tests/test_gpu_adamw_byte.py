"""The AdamW step with moments in 8 bits against its fp64 reference.

Bounds (e = 2^-24, every fp32 operation rounds once):
  m, v   two products with a rounded constant and a sum each: off by 3 e of the sum of their terms'
         magnitudes, v, whose terms are positive and whose square rounds too, by 4 e of itself;
  param  mhat / (sqrt(vhat) + eps): 2 e more on mhat, half of v's and 5 e of root, sum and
         quotient; p (1 - lr wd) - lr update: 4 e of p and 2 e of the update's product.  With m's
         terms of opposite signs its error is relative to the terms, not to m.
A moment's value then lies on the grid at floor(place + fraction).  The place's relative error is
that of the moment and one more rounding, so where place + fraction is nearer to a whole number
than 8 e of the place (16 at most, in grid units) and 2^-20 for the sum's own rounding, either
neighbour is right; elsewhere one is.  A block's scale may be one binade off only where its
largest value lies within 8 e of a power of two.
"""
import numpy as np
import pytest

from oracle import adamw_byte as ref

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
HP = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _np(t):
    return t.double().cpu().numpy()


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _shift(t, offset):
    """A copy of t that starts `offset` elements into its memory."""
    raw = torch.zeros(t.numel() + offset, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=DEV)
    view = raw[offset:].view(t.shape)
    view.copy_(t.view(torch.uint8) if t.element_size() == 1 else t)
    return view.view(t.dtype)


def _segment(n, seed, grad_type=torch.float32, copy_type=None, offset=0, warm=2):
    """A tensor whose moments come from steps of their own; rows of very different sizes."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    size = torch.exp(3 * torch.randn(-(-n // 64), 1, generator=g, device=DEV)).expand(-1, 64).reshape(-1)[:n]
    p = torch.randn(n, generator=g, device=DEV)
    state = ma.adamw_byte_state(p)
    for t in range(1, warm + 1):
        grad = torch.randn(n, generator=g, device=DEV) * size
        ma.adamw_byte_step_multi([(p, grad, *state)], step=t, seed=seed, **HP)
    grad = (torch.randn(n, generator=g, device=DEV) * size * (torch.rand(n, generator=g, device=DEV) < 0.9)).to(grad_type)
    copy = None if copy_type is None else torch.zeros(n, dtype=copy_type, device=DEV)
    seg = (p, grad, *state, copy)
    return tuple(t if t is None else _shift(t, offset) for t in seg)


def _reference(seg, step, **hp):
    p, g, m, ms, v, vs = (_np(t) if i not in (3, 5) else _bytes(t) for i, t in enumerate(seg[:6]))
    m, v = ref.widen(m, ms), ref.widen(v, vs)
    return (p, g, m, v), ref.step(p, g, m, v, step=step, **{**HP, **hp})


def _check_moment(value, scale, x, err, kind, fraction, floor):
    """value, scale: the kernel's; x: the reference's moment, off by err."""
    e, got = ref.exponents(x, kind), _bytes(scale).astype(np.int64) - 127
    big = np.abs(ref.blocks(x)).max(1)
    near = np.abs(big / np.exp2(np.round(np.log2(np.maximum(big, 1e-300)))) - 1) <= 8 * E
    assert ((got == e) | (near & (np.abs(got - e) <= 1))).all()
    place, unit = ref.places(x, got, kind)
    size = np.exp2(got.astype(np.float64)).repeat(ref.BLOCK)[:place.size]
    raw = np.abs(place) + fraction
    slack = err / (unit * size) + 2 * E * np.abs(place) + 2.0 ** -20
    low, high = np.floor(raw - slack), np.floor(raw + slack)
    if floor:
        low, high = (np.where((x > 0) & (t <= 0), 1, t) for t in (low, high))
    q = np.abs(_np(value)) / unit
    # at the border of a binade the grid below is half as wide
    assert ((q >= np.minimum(low, high)) & (q <= high) | (np.abs(q * 2 - np.round(q * 2)) == 0) & (np.abs(q - raw) <= 1)).all()
    exact = low == high
    assert exact.mean() > 0.99
    assert (q[exact] == high[exact]).all()
    sign = np.sign(_np(value))
    # a moment whose terms cancel to less than its error may have either sign
    assert ((sign == np.sign(x)) | (sign == 0) | (np.abs(x) <= err)).all()


def _check(before, after, step, first, seed, **hp):
    (p, g, m, v), (rp, rm, rv) = _reference(before, step, **hp)
    b1, b2 = HP["beta1"], HP["beta2"]
    if not hp.get("decoupled", True):
        g = g + HP["weight_decay"] * p
    terms = np.abs(b1 * m) + np.abs((1 - b1) * g)
    em, ev = 4 * E * terms, 6 * E * rv
    root = np.sqrt(rv / (1 - b2 ** step)) + HP["eps"]
    upd = np.abs(rm / (1 - b1 ** step) / root)
    bound = 6 * E * np.abs(p) + HP["lr"] * (em / (1 - b1 ** step) / root + 16 * E * upd)
    got = _np(after[0])
    assert (np.abs(got - rp) <= bound * 1.01 + 2.0 ** -140).all()
    fm, fv = ref.fractions(first, p.size, seed, step)
    _check_moment(after[2], after[3], rm, em, ref.E4M3, fm, False)
    _check_moment(after[4], after[5], rv, ev, ref.E5M2, fv, True)
    if after[6] is not None:
        assert torch.equal(after[6], after[0].to(after[6].dtype))


def _clone(segs):
    return [tuple(t if t is None else t.view(torch.uint8).clone().view(t.dtype) if t.element_size() == 1 else t.clone()
                  for t in s) for s in segs]


def _same(a, b):
    return all((x is None and y is None) or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for s, t in zip(a, b) for x, y in zip(s, t))


@pytest.mark.parametrize("n", [1, 3, 63, 64, 65, 1000, 4095, 4096, 4097, 70001])
@pytest.mark.parametrize("grad_type,copy_type", [(torch.float32, None), (torch.bfloat16, torch.bfloat16),
                                                 (torch.float16, torch.float16), (torch.float32, torch.bfloat16)])
def test_step(n, grad_type, copy_type):
    seed = 2 ** 33 + n
    before = _segment(n, n, grad_type, copy_type)
    after, = _clone([before])
    ma.adamw_byte_step_multi([after], step=3, seed=seed, **HP)
    _check(before, after, 3, 0, seed)


@pytest.mark.parametrize("hp", [dict(decoupled=False), dict(cautious_wd=True)])
def test_decay(hp):
    before = _segment(5000, 5)
    after, = _clone([before])
    ma.adamw_byte_step_multi([after], step=7, seed=1, **HP, **hp)
    _check(before, after, 7, 0, 1, **hp)


@pytest.mark.parametrize("sizes", [[5, 0, 64, 129, 5000], [100 + 37 * i for i in range(100)]])
def test_many_tensors(sizes):
    """Over several launches; every tensor's numbers start at a multiple of 64."""
    before = [_segment(max(n, 1), i, torch.bfloat16 if i % 3 else torch.float32,
                       torch.bfloat16 if i % 2 else None, offset=i % 5) for i, n in enumerate(sizes)]
    before = [s if n else tuple(t if t is None else t[:0] for t in s) for s, n in zip(before, sizes)]
    after = _clone(before)
    ma.adamw_byte_step_multi(after, step=4, seed=9, **HP)
    first = 0
    for b, a, n in zip(before, after, sizes):
        if n:
            _check(b, a, 4, first, 9)
        first += -(-n // 64) * 64


def test_elements_behind_2_32():
    """Their addresses and their numbers pass 32 bits."""
    n, seed, warm = (1 << 32) + 130, 21, 2
    start = (1 << 32) - 128
    p = torch.zeros(n, device=DEV)
    grad = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    seg = (p, grad, *ma.adamw_byte_state(p), torch.zeros(n, dtype=torch.bfloat16, device=DEV))
    tail = tuple(t[start // 64:] if i in (3, 5) else t[start:] for i, t in enumerate(seg))
    g = torch.Generator(device=DEV).manual_seed(5)
    tail[0].copy_(torch.randn(n - start, generator=g, device=DEV))
    for t in range(1, warm + 2):
        tail[1].copy_(torch.randn(n - start, generator=g, device=DEV))
        before, = _clone([tail])
        ma.adamw_byte_step_multi([seg], step=t, seed=seed, **HP)
        _check(before, tail, t, start, seed)
    assert not p[:start].any() and not seg[4].view(torch.uint8)[:start].any()


@pytest.mark.parametrize("n", [65, 5003])
def test_alignment_changes_nothing(n):
    runs = []
    for offset in (0, 1, 2, 3):
        seg, = [_segment(n, 3, torch.float16, torch.bfloat16, offset=offset)]
        again, = _clone([seg])
        ma.adamw_byte_step_multi([seg], step=3, seed=4, **HP)
        ma.adamw_byte_step_multi([again], step=3, seed=4, **HP)
        assert _same([seg], [again])
        runs.append(_clone([seg]))
    assert all(_same(runs[0], r) for r in runs[1:])


def test_neighbours_of_a_tensor_are_left_alone():
    n, pad = 1001, 64
    seg = _segment(n, 8, torch.float32, torch.bfloat16)
    wide = []
    for t in seg:
        raw = torch.full((t.numel() + 2 * pad,), 77, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=DEV)
        raw[pad:-pad].copy_(t.view(torch.uint8) if t.element_size() == 1 else t)
        wide.append((raw, raw[pad:-pad].view(t.dtype)))
    ma.adamw_byte_step_multi([tuple(v for _, v in wide)], step=3, seed=2, **HP)
    for raw, _ in wide:
        assert (raw[:pad] == 77).all() and (raw[-pad:] == 77).all()


def test_rounding_is_unbiased():
    """One element's step in 2^20 copies, whose moments lie between two values of their types."""
    n = 1 << 20
    p, grad = torch.zeros(n, device=DEV), torch.full((n,), 0.37, device=DEV)
    seg = (p, grad, *ma.adamw_byte_state(p))
    ma.adamw_byte_step_multi([seg], step=1, seed=5, **HP)
    for value, scale, want in ((seg[2], seg[3], 0.37 * (1 - HP["beta1"])), (seg[4], seg[5], 0.37 ** 2 * (1 - HP["beta2"]))):
        got = _np(ma.adamw_byte_values(value, scale))
        near = np.unique(got)
        assert near.size == 2 and near[0] < want < near[1]
        # the mean of n coins; the grid of 2^16 fractions adds at most one of them
        assert abs(got.mean() - want) <= (near[1] - near[0]) * (5 * 0.5 / n ** 0.5 + 2.0 ** -16)


def test_slow_averages_move():
    """Without a gradient exp_avg_sq falls by a factor beta2 a step, which no rounding to nearest
    would let it.  Each step's rounding moves an element by at most a quarter of itself with
    probability (1 - beta2) / 0.125 at most, so the product of 400 steps has a relative deviation
    below sqrt(400 0.25^2 0.016) = 0.64 per element, and its mean over 2^16 one of 0.0025."""
    n, beta2 = 1 << 16, 0.998
    p, zero = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    state = ma.adamw_byte_state(p)
    ma.adamw_byte_step_multi([(p, torch.ones(n, device=DEV), *state)], step=1, lr=0.0, beta2=beta2)
    start = _np(ma.adamw_byte_values(state[2], state[3])).mean()
    for t in range(2, 402):
        ma.adamw_byte_step_multi([(p, zero, *state)], step=t, lr=0.0, beta2=beta2, seed=11)
    got = _np(ma.adamw_byte_values(state[2], state[3])).mean()
    assert abs(got / (start * beta2 ** 400) - 1) < 5 * 0.0025 * 1.2


def test_no_gradient_and_no_state():
    """Zero moments and gradients stay zero; the parameter decays only."""
    p = torch.randn(200, device=DEV)
    keep = p.clone()
    state = ma.adamw_byte_state(p)
    ma.adamw_byte_step_multi([(p, torch.zeros(200, device=DEV), *state)], step=1, **HP)
    assert (_np(state[0].float()) == 0).all() and (_np(state[2].float()) == 0).all()
    scale = np.float32(1) - np.float32(HP["lr"]) * np.float32(HP["weight_decay"])
    assert torch.allclose(p, keep * float(scale), rtol=2 ** -23, atol=0)


def test_a_positive_second_moment_stays_positive():
    """Next to a value 2^40 times as large an element's exp_avg_sq is far below its type's least."""
    p = torch.zeros(64, device=DEV)
    grad = torch.full((64,), 1e-12, device=DEV)
    grad[5] = 1.0
    state = ma.adamw_byte_state(p)
    ma.adamw_byte_step_multi([(p, grad, *state)], step=1, **HP)
    assert (_np(state[2].float()) > 0).all()
    ma.adamw_byte_step_multi([(p, grad, *state)], step=2, **HP)
    assert (np.abs(_np(p)) <= 2 * 2 * HP["lr"]).all()


def test_not_a_number_stays_in_its_element():
    n = 256
    p, grad = torch.ones(n, device=DEV), torch.full((n,), 0.5, device=DEV)
    grad[70], grad[130], grad[140] = float("nan"), float("inf"), -float("inf")
    clean = torch.full((n,), 0.5, device=DEV)
    a, b = (p, grad, *ma.adamw_byte_state(p)), (p.clone(), clean, *ma.adamw_byte_state(p))
    for s in (a, b):
        ma.adamw_byte_step_multi([s], step=1, **HP)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[[70, 130, 140]] = True
    assert not torch.isfinite(a[0][bad]).any()
    assert torch.equal(a[0][~bad], b[0][~bad])
    assert not torch.isfinite(a[2].float()[bad]).any() and not torch.isfinite(a[4].float()[bad]).any()
    # block 1 holds the NaN: its other elements are as without it
    assert _same([(a[2][64:128][~bad[64:128]],)], [(b[2][64:128][~bad[64:128]],)])
    assert torch.isfinite(a[2].float()[~bad]).all()


def test_versions_and_streams():
    seg = _segment(500, 2, torch.bfloat16, torch.bfloat16)
    ref_seg, = _clone([seg])
    versions = [t._version for t in seg]
    ma.adamw_byte_step_multi([ref_seg], step=3, seed=1, **HP)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ma.adamw_byte_step_multi([seg], step=3, seed=1, stream=side, **HP)
    torch.cuda.current_stream().wait_stream(side)
    assert _same([seg], [ref_seg])
    assert [t._version - v for t, v in zip(seg, versions)] == [1, 0, 1, 1, 1, 1, 1]


def test_captured_step():
    seg = _segment(3000, 4, torch.bfloat16, torch.bfloat16)
    eager, = _clone([seg])
    start, = _clone([seg])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ma.adamw_byte_step_multi([seg], step=3, seed=1, **HP)
    ma.adamw_byte_step_multi([eager], step=3, seed=1, **HP)
    for _ in range(3):
        for t, s in zip(seg, start):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        assert _same([seg], [eager])
        torch.randn(1000, device=DEV).sum().item()


# ---------------------------------------------------------------- in the optimizer
def _group(shapes, draw, **kw):
    g = torch.Generator(device=DEV).manual_seed(draw)
    params = [torch.nn.Parameter(torch.randn(s, generator=g, device=DEV)) for s in shapes]
    return params, dict({"kind": "adamw", "params": params, "lr": 1e-2, "betas": (0.9, 0.95), "state_bits": 8}, **kw)


def test_optimizer_steps_as_the_call():
    shapes = [(30, 20), (65,), (7,)]
    params, group = _group(shapes, 1, weight_decay=0.1, seed=6)
    copy = torch.zeros(30, 20, dtype=torch.bfloat16, device=DEV)
    opt = ma.MuonAdamW([dict(group, copies=[copy, None, None])])
    assert 2.0 < opt.state_bytes_per_param("adamw") < 2.1
    mine = [(p.data.clone(), None, *ma.adamw_byte_state(p)) for p in params]
    for t in range(1, 4):
        grads = [torch.randn(s, device=DEV) for s in shapes]
        for p, gr in zip(params, grads):
            p.grad = gr
        if t == 2:
            params[1].grad = None  # not stepped
        opt.step()
        live = [i for i in range(3) if t != 2 or i != 1]
        ma.adamw_byte_step_multi([(mine[i][0], grads[i], *mine[i][2:]) for i in live], step=t, lr=1e-2, beta1=0.9,
                                 beta2=0.95, weight_decay=0.1, seed=6)
        assert all(torch.equal(p.data, m[0]) for p, m in zip(params, mine))
        assert torch.equal(copy, params[0].data.to(torch.bfloat16))


def test_optimizer_state_moves_to_another():
    params, group = _group([(40, 33), (5,)], 2)
    opt = ma.MuonAdamW([group])
    grads = [[torch.randn_like(p) for p in params] for _ in range(2)]
    for p, g in zip(params, grads[0]):
        p.grad = g
    opt.step()
    twins = [torch.nn.Parameter(p.data.clone()) for p in params]
    other = ma.MuonAdamW([dict(group, params=twins)])
    other.load_state_dict(opt.state_dict())
    for p, q, g in zip(params, twins, grads[1]):
        p.grad, q.grad = g, g.clone()
    opt.step()
    other.step()
    assert all(torch.equal(p.data, q.data) for p, q in zip(params, twins))
    wide = ma.MuonAdamW([dict(group, params=[torch.nn.Parameter(p.data.clone()) for p in params], state_bits=32)])
    for a, b in ((wide, opt), (opt, wide)):
        with pytest.raises(ValueError, match="bits"):
            a.load_state_dict(b.state_dict())


def test_optimizer_takes_token_gradients():
    (table,), group = _group([(50, 24)], 3)
    opt = ma.MuonAdamW([group])
    twin = torch.nn.Parameter(table.data.clone())
    dense = ma.MuonAdamW([dict(group, params=[twin])])
    tokens = torch.randint(0, 50, (40,), device=DEV)
    out = ma.embedding(tokens, table, optimizer=opt)
    w = torch.randn_like(out)
    (out * w).sum().backward()
    (ma.embedding(tokens, twin) * w).sum().backward()
    opt.step()
    dense.step()
    assert torch.equal(table.data, twin.data)
