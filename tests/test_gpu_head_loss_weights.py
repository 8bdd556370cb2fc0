"""The head loss's row weights: their scaling before g is rounded, and rows of weight zero.

Bounds: as derived in test_gpu_head_loss.  The scaling is a power of two made of the largest finite
weight of a row with a target, so that it rounds nothing itself.
"""
import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

from test_gpu_head_loss import DEV, TYPES, _inputs, _near, _reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim", [(300, 136), (300, 1100), (40, 136), (90, 200)])
def test_rows_do_not_depend_on_the_largest_weight(dtype, n, dim):
    """The row of the largest weight loses its target: the others' dh keep their bits.  (In fp16 the
    scaling decides which values of g are below the least normal number: there within the bound.)"""
    h, w, labels, rw = _inputs(n, 700, dim, dtype, 21, ignored=0)
    rw[1] = 1.7
    on = torch.arange(n, device=DEV) != 1
    rest = labels.clone()
    rest[1] = -100
    calls = [lambda l: ma.head_loss_grad(h, w, l, rw)[1]]
    lse = ma.head_loss_forward(h, w, labels)[1]
    calls.append(lambda l: ma.head_loss_backward(h, w, l, lse, rw)[0])
    for call in calls:
        with_it, without = call(labels), call(rest)
        assert not without[1].any()
        if dtype != torch.float16:
            assert torch.equal(with_it[on], without[on])
    ref = _reference(h, w, rest, rw)
    _near(ma.head_loss_grad(h, w, rest, rw)[1], ref[4], ref[6])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weight,size", [(1e-6, 1.0), (2e5, 1e-3)])
@pytest.mark.parametrize("n", [40, 150])
def test_an_infinite_weight_leaves_other_rows_their_bounds(dtype, weight, size, n):
    """Small weights do not vanish in 16 bits next to it, nor do large ones overflow."""
    h, w, labels, rw = _inputs(n, 400, 72, dtype, 12, ignored=0)
    w = (w.float() * size).to(dtype)
    rw = rw * weight
    on = torch.arange(n, device=DEV) != 17
    ref = _reference(h, w, labels, torch.where(on, rw, 0.0))
    rw[17] = float("inf")
    lse = ma.head_loss_forward(h, w, labels)[1]
    ref_lse = _reference(h, w, labels, torch.where(on, rw, 0.0), lse)
    for dh, (want, bound) in ((ma.head_loss_grad(h, w, labels, rw)[1], (ref[4], ref[6])),
                              (ma.head_loss_backward(h, w, labels, lse, rw)[0], (ref_lse[4], ref_lse[6]))):
        assert not torch.isfinite(dh[17]).any()
        _near(dh[on], want[on], bound[on])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim", [(1, 136), (40, 136), (40, 1100), (100, 136), (300, 136), (300, 1100)])
def test_an_infinity_in_the_weight_beside_rows_of_weight_zero(dtype, n, dim):
    """An entry of the vocabulary whose logits are all -inf has probability 0: it takes part in nothing,
    its own gradient is 0, and so is dh of a row of weight 0.  (The others' dh has 0 x inf in one
    column.)  fp32 above 128 rows takes no infinities."""
    if dtype == torch.float32 and n > 128:
        pytest.skip("magnitudes up to 2^127")
    h, w, labels, rw = _inputs(n, 700, dim, dtype, 4, ignored=0)
    h[:, 3] = -h[:, 3].abs() - 0.125
    labels[labels == 5] = 6
    rw[n // 2] = 0.0
    ref = _reference(h, torch.cat([w[:5], w[6:]]), labels - (labels > 5).long(), rw)
    w[5, 3] = float("inf")
    cols = torch.arange(dim, device=DEV) != 3
    entries = torch.arange(700, device=DEV) != 5
    loss, dh, dw = ma.head_loss_grad(h, w, labels, rw)
    _near(loss, ref[0], ref[2])
    lse = ma.head_loss_forward(h, w, labels)[1]
    ref_lse = _reference(h, torch.cat([w[:5], w[6:]]), labels - (labels > 5).long(), rw, lse)
    for got, want in (((dh, dw), ref), (ma.head_loss_backward(h, w, labels, lse, rw), ref_lse)):
        assert not got[0][n // 2].any() and not got[1][5].any()
        _near(got[0][:, cols], want[4][:, cols], want[6][:, cols])
        _near(got[1][entries], want[5], want[7])
