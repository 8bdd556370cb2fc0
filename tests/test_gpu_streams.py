"""The optimizer calls' own workspaces when a stream is given."""
import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_workspaces_are_the_streams_own_memory(monkeypatch):
    """A call's workspace on another stream is not the one that a call on the current stream,
    whose work that stream does not wait for, has just dropped; both give what they give alone."""
    from adamw_optimizer_step_muon_amd import _lib

    g = torch.Generator(device=DEV).manual_seed(1)
    a, b = (torch.randn(4, 256, 512, generator=g, device=DEV) for _ in "ab")
    want = [torch.empty_like(a) for _ in "ab"]
    for x, y in zip((a, b), want):
        ma.newton_schulz(x, y)
    got = [torch.empty_like(a) for _ in "ab"]
    steps = [[t.clone() for t in (a, b, torch.zeros_like(a))] for _ in range(3)]
    torch.cuda.synchronize()
    seen, scratch = [], _lib._scratch

    def spy(nbytes, device, stream):
        ws = scratch(nbytes, device, stream)
        seen.append((stream is None, ws.data_ptr()))
        return ws

    monkeypatch.setattr(_lib, "_scratch", spy)
    side, big = torch.cuda.Stream(), torch.randn(2048, 2048, generator=g, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        big = torch.tanh(big @ big)  # the current stream has work to come first
    ma.newton_schulz(a, got[0])
    ma.newton_schulz(b, got[1], stream=side)
    for s, stream in zip(steps, (None, side, None)):
        ma.muon_step([s], lr=0.02, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for s in steps[1:]:
        assert all(torch.equal(p, q) for p, q in zip(s, steps[0]))
    here, there = ({p for k, p in seen if k == own} for own in (True, False))
    assert len(seen) == 5 and not here & there
