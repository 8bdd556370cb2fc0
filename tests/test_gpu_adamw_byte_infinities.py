"""Infinities in the AdamW step with moments in 8 bits stay in their elements.

An element's random bits come from its number, seed and step, and its block's scale from the block's
largest finite magnitude: so all elements but the infinite ones are, bit for bit, what they are in a
run in which those have a zero gradient.
"""
import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HP = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
INF = float("inf")


def _bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int32)


def _runs(n, places, dtype, steps=3):
    """Two runs, the second with zeros at `places` {element: gradient of the first step}, stepped
    three times; yields (step, with, without)."""
    g = torch.Generator(device=DEV).manual_seed(n)
    p = torch.randn(n, generator=g, device=DEV)
    a, b = ((p.clone(), *ma.adamw_byte_state(p)) for _ in range(2))
    for step in range(1, steps + 1):
        grad = torch.randn(n, generator=g, device=DEV).to(dtype)
        for s, put in ((a, True), (b, False)):
            mine = grad.clone()
            for at, value in places.items():
                mine[at] = value if put and step == 1 else 0.0
            ma.adamw_byte_step_multi([(s[0], mine, *s[1:])], step=step, seed=5, **HP)
        yield step, a, b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,places", [(320, {70: float("nan"), 130: INF, 140: -INF, 191: INF, 319: INF}),
                                      (67, {66: INF}), (5, {0: -INF}), (4096 + 64, {4096: INF, 17: -INF})])
def test_neighbours_go_on(n, places, dtype):
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[list(places)] = True
    for step, a, b in _runs(n, places, dtype):
        for t, u in ((a[0], b[0]), (a[1], b[1]), (a[3], b[3])):
            assert torch.equal(_bits(t)[~bad], _bits(u)[~bad]), step
            assert not torch.isfinite(t.float()[bad]).any(), step
        for t, u in ((a[2], b[2]), (a[4], b[4])):  # scales
            assert torch.equal(_bits(t), _bits(u)), step


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_square_that_overflows(dtype):
    """1e20 is finite, its square is not: exp_avg_sq is infinite in that element alone.  (Its exp_avg
    is finite, and sets its block's scale.)"""
    bad = torch.zeros(192, dtype=torch.bool, device=DEV)
    bad[100] = True
    for step, a, b in _runs(192, {100: 1e20}, dtype):
        assert torch.isinf(a[3].float()[bad]).all()
        assert torch.equal(_bits(a[3])[~bad], _bits(b[3])[~bad]) and torch.equal(_bits(a[4]), _bits(b[4])), step
        out = torch.ones(192, dtype=torch.bool, device=DEV)
        out[64:128] = False
        assert torch.equal(_bits(a[1])[out], _bits(b[1])[out]) and torch.equal(a[0][out], b[0][out])
        if step == 1:
            assert torch.equal(a[0][~bad], b[0][~bad])


def test_a_block_of_infinities():
    for step, a, b in _runs(192, {i: INF for i in range(64, 128)}, torch.float32, steps=2):
        assert not torch.isfinite(a[1].float()[64:128]).any() and not torch.isfinite(a[3].float()[64:128]).any()
        out = torch.ones(192, dtype=torch.bool, device=DEV)
        out[64:128] = False
        for t, u in ((a[0], b[0]), (a[1], b[1]), (a[3], b[3])):
            assert torch.equal(_bits(t)[out], _bits(u)[out])
