"""The head loss's calls in workspaces of exactly the size that each asks for: whatever the memory held, they
give the same bits as with one of their own, and leave what lies behind it as it was."""
import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

from test_gpu_head_loss import DEV, SIZES, TYPES, _inputs  # noqa: E402

pytestmark = pytest.mark.gpu
BEHIND = 1 << 20


@pytest.mark.parametrize("n,vocab,dim", SIZES + [(200, 20001, 72), (33, 30000, 600), (600, 9000, 1280)])
@pytest.mark.parametrize("dtype", TYPES)
def test_calls_stay_within_their_workspace(n, vocab, dim, dtype):
    h, w, labels, rw = _inputs(n, vocab, dim, dtype, n + dim)
    lse = ma.head_loss_forward(h, w, labels)[1]
    calls = {"forward": lambda **kw: ma.head_loss_forward(h, w, labels, **kw),
             "backward": lambda **kw: ma.head_loss_backward(h, w, labels, lse, rw, **kw),
             "grad": lambda **kw: ma.head_loss_grad(h, w, labels, rw, **kw)}
    for name, call in calls.items():
        want = call()
        need = ma.head_loss_workspace_bytes(h, w, call=name)
        raw = torch.full((need + BEHIND,), 255, dtype=torch.uint8, device=DEV)  # NaN in every type
        got = call(workspace=raw[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        assert (raw[need:] == 255).all(), name
        with pytest.raises(ma.MuonAdamWError, match="workspace"):
            call(workspace=raw[:need - 1])
