"""The head loss's workspace sizes, which are made on the host (no GPU needed)."""
import random

import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

from adamw_optimizer_step_muon_amd import _lib  # noqa: E402

F32, F16, BF16 = 0, 1, 2
FORWARD, ANY = 0, 1


def _bytes(type_, n, dim, vocab, calls, stride=None):
    return _lib.load().ma_head_loss_workspace_bytes(type_, n, dim, vocab, 256, stride or dim, calls)


def _sizes(count):
    rng = random.Random(7)
    for _ in range(count):
        yield rng.randrange(3), int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 18))


def test_the_default_size_serves_the_forward_call():
    sizes = [(F32, 52, 4488, 66709), (BF16, 8, 4096, 32000), *_sizes(3000)]
    for type_, n, dim, vocab in sizes:
        assert _bytes(type_, n, dim, vocab, ANY) >= _bytes(type_, n, dim, vocab, FORWARD) > 0, (type_, n, dim, vocab)


def test_the_helper_has_the_same_default():
    h, w = torch.empty(52, 4488), torch.empty(66709, 4488)
    assert ma.head_loss_workspace_bytes(h, w) >= ma.head_loss_workspace_bytes(h, w, gradients=False)


BACKWARD, GRAD = 2, 3
MB = 1 << 20


def test_any_call_is_the_largest():
    for size in _sizes(1000):
        each = [_bytes(*size, calls) for calls in (FORWARD, BACKWARD, GRAD)]
        assert _bytes(*size, ANY) == max(each) and min(each) > 0


@pytest.mark.parametrize("type_,n,dim,vocab", [(BF16, 2048, 1280, 65536), (F16, 2048, 1280, 65536), (F32, 511, 768, 65536)])
def test_the_backward_call_has_no_room_for_logits(type_, n, dim, vocab):
    """Its logits become g at once; those of the call for both directions are kept beside g."""
    rows = -(-n // 256) * 256
    assert _bytes(type_, n, dim, vocab, GRAD) - _bytes(type_, n, dim, vocab, BACKWARD) >= rows * vocab * 4


def test_kept_fp32_logits_become_g():
    """In place, on the fp32 instructions.  (100 rows take 128; up to 64 parts of dhidden.)"""
    rows, dim, vocab = 128, 256, 40000
    assert _bytes(F32, 100, dim, vocab, GRAD) <= rows * (vocab + 256) * 4 + 64 * rows * dim * 4 + rows * dim * 4 + MB


@pytest.mark.parametrize("type_,value", [(F32, 4), (F16, 2), (BF16, 2)])
def test_few_rows_take_the_memory_of_few(type_, value):
    """One row: g and kept logits (the same memory in fp32) of one tile of 32 or 64 rows, and up to 64 parts
    of dhidden."""
    rows, vocab, dim = 32 if type_ == F32 else 64, 128000, 2048
    room = rows * (vocab + 256) * (4 if type_ == F32 else value + 4) + 64 * rows * dim * 4 + rows * dim * value
    assert _bytes(type_, 1, dim, vocab, GRAD) <= room + MB
    assert _bytes(type_, 1, dim, vocab, FORWARD) <= rows * (vocab + 256) * 4 * 8 + rows * dim * value + MB


def test_the_helper_names_the_calls():
    h, w = torch.empty(52, 448), torch.empty(6670, 448)
    got = {call: ma.head_loss_workspace_bytes(h, w, call=call) for call in ("forward", "backward", "grad")}
    assert got == {call: _bytes(F32, 52, 448, 6670, k) for call, k in (("forward", 0), ("backward", 2), ("grad", 3))}
    with pytest.raises(ValueError, match="call"):
        ma.head_loss_workspace_bytes(h, w, call="both")
