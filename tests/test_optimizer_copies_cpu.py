"""The 16-bit copies of a group with 8-bit moments follow a restored checkpoint (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_copies_follow_a_restored_state(dtype):
    """Restored parameters, then the optimizer: what a head reads before the next step is the restored
    weight, not the one before."""
    g = torch.Generator().manual_seed(3)
    params = [torch.nn.Parameter(torch.randn(s, generator=g)) for s in ((6, 4), (5,), (3,))]
    copies = [torch.zeros(24, dtype=dtype), None, torch.zeros(3, dtype=dtype)]
    opt = ma.MuonAdamW([{"kind": "adamw", "params": params, "state_bits": 8, "copies": copies}])
    saved, state = [p.detach().clone() for p in params], opt.state_dict()
    assert "copies" not in state["param_groups"][0]
    with torch.no_grad():
        for p, c in zip(params, copies):
            p.add_(1.0)
            if c is not None:
                c.copy_(p.reshape(c.shape))
        for p, s in zip(params, saved):
            p.copy_(s)
    versions = [None if c is None else c._version for c in copies]
    opt.load_state_dict(state)
    for p, c, version in zip(params, copies, versions):
        if c is not None:
            assert torch.equal(c, p.detach().reshape(c.shape).to(dtype)) and c._version > version
