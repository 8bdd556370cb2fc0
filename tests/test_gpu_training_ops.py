"""The training operators as they are used together: a small model's training steps with
MuonAdamW, graph capture, other streams and concurrent calls."""
import threading

import pytest

torch = pytest.importorskip("torch")
ma = pytest.importorskip("adamw_optimizer_step_muon_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, D, T, K, EPS = 97, 32, 40, 6, 1e-5
TAU, SCALE = 2.0, D ** 0.5


def _model(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return {"table": 0.2 * r(V, D), "g0": 1 + 0.1 * r(D), "b0": 0.1 * r(D), "hidden": 0.2 * r(D, D),
            "g1": 1 + 0.1 * r(D), "head": 0.2 * r(V, D)}


def _batch(seed):
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)
    tokens = torch.randint(0, V, (4, T // 4), generator=g, device=DEV)
    tokens[2, 7:] = -1  # padded sequence
    ids = torch.randint(0, V, (4, T // 4, K), generator=g, device=DEV)
    ids[2, 7:] = -1
    return tokens, torch.randn(4, T // 4, K, generator=g, device=DEV), ids


def _loss(p, batch, optimizer=None):
    tokens, teacher, ids = batch
    x = ma.embedding(tokens, p["table"], scale=SCALE, optimizer=optimizer)
    h = ma.layer_norm(x, p["g0"], p["b0"], eps=EPS)
    x = x + torch.tanh((h.view(-1, D) @ p["hidden"]).view(x.shape))
    y = ma.layer_norm(x, p["g1"], eps=EPS)
    logits = (y.view(-1, D) @ p["head"].t()).view(*tokens.shape, V)
    return ma.distill_loss(logits, teacher, ids, temperature=TAU).mean()


def _plain_loss(p, batch):
    """The same model in fp64 torch operations."""
    tokens, teacher, ids = batch

    def norm(x, w, b=0.0):
        c = x - x.mean(-1, keepdim=True)
        return c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * w + b

    live = tokens >= 0
    x = torch.where(live[..., None], p["table"][tokens.clamp(min=0)] * SCALE, 0.0)
    x = x + torch.tanh((norm(x, p["g0"], p["b0"]).view(-1, D) @ p["hidden"]).view(x.shape))
    logits = (norm(x, p["g1"]).view(-1, D) @ p["head"].t()).view(*tokens.shape, V)
    log_q = torch.log_softmax(logits / TAU, -1)
    log_p = torch.log_softmax(teacher.double() / TAU, -1)
    kl = (log_p.exp() * (log_p - log_q.gather(-1, ids.clamp(min=0)))).sum(-1)
    return TAU ** 2 * torch.where(live, kl, 0.0).mean()


def _leaves(p):
    return {k: t.clone().requires_grad_(True) for k, t in p.items()}


def test_gradients_of_a_model():
    """Every parameter's gradient against torch's fp64 one.  Ten stages of at most 130
    roundings each (sums of 32, 40 or 97 terms): 1300 * 2^-24 = 8e-5 of the terms."""
    p, batch = _model(1), _batch(1)
    own, plain = _leaves(p), {k: t.double().requires_grad_(True) for k, t in p.items()}
    a, b = _loss(own, batch), _plain_loss(plain, batch)
    a.backward(), b.backward()
    assert abs(float(a.detach()) - float(b.detach())) <= 8e-5 * abs(float(b.detach()))
    for k in p:
        d = (own[k].grad.double() - plain[k].grad).norm() / plain[k].grad.norm()
        assert d <= 8e-5, (k, float(d))
    assert own["table"].grad[batch[0].unique()[1:]].any()


def _optimizer(p):
    return ma.MuonAdamW([{"kind": "muon", "params": [p["hidden"]], "lr": 0.02},
                         {"kind": "adamw", "params": [p[k] for k in ("table", "g0", "b0", "g1", "head")],
                          "lr": 1e-2, "weight_decay": 0.1}])


@pytest.mark.parametrize("micro", [1, 2])
def test_steps_with_token_gradients_are_bitwise_the_dense_ones(micro):
    """Three steps of `micro` batches each; two batches add up in a dense gradient, one is
    stepped from the tokens."""
    runs = []
    for by_token in (False, True):
        p = _leaves(_model(2))
        opt = _optimizer(p)
        for step in range(3):
            for i in range(micro):
                _loss(p, _batch(10 * step + i), opt if by_token else None).backward()
            assert (p["table"].grad is None) == by_token
            opt.step()
            opt.zero_grad()
            assert p["table"].grad is None
        runs.append((p, opt.state_dict()["state"]))
    for k in runs[0][0]:
        # the two batches' dense gradients are added elementwise by autograd, and by the
        # accumulating kernel: the same one rounding
        assert torch.equal(runs[0][0][k], runs[1][0][k]), k
    for i, st in runs[0][1].items():
        for k in st:
            assert torch.equal(st[k], runs[1][1][i][k])


def test_tied_table_adds_token_and_dense_gradients():
    p = _leaves(_model(3))
    opt = _optimizer(p)
    tokens, dout = torch.tensor([3, 3, 5], device=DEV), torch.randn(3, D, device=DEV)
    dense = torch.randn(V, D, device=DEV)
    p["table"].grad = dense.clone()
    opt.add_token_gradient(p["table"], tokens, dout, 2.0)
    before = p["table"].detach().clone()
    opt.step()
    want = dense + ma.embedding_backward(dout, tokens, V, scale=2.0)
    assert torch.equal(p["table"].grad, want)
    q = [before, want, torch.zeros_like(want), torch.zeros_like(want)]
    ma.adamw_step(*q, step=1, lr=1e-2, weight_decay=0.1)
    assert torch.equal(p["table"], q[0])


def _calls(s):
    """One training step's calls on static buffers."""
    x = ma.embedding_forward(s["table"], s["tokens"], scale=SCALE, out_dtype=torch.bfloat16)
    y, mean, rstd = ma.layer_norm_forward(x, s["g"], s["b"])
    logits = y @ s["head"]
    loss, dlogits = ma.distill_loss_grad(logits, s["teacher"], s["ids"], s["w"], temperature=TAU)
    stats = ma.distill_forward(logits, s["teacher"], s["ids"], temperature=TAU)[1]
    dlogits2 = ma.distill_backward(logits, s["teacher"], s["ids"], stats, s["w"], temperature=TAU)
    dy = dlogits @ s["head_t"]
    dx, dg, db = ma.layer_norm_backward(dy, x, mean, rstd, s["g"])
    grad = ma.embedding_backward(dx, s["tokens"], s["table"].shape[0], scale=SCALE)
    ma.adamw_step_embedding(s["p"], s["tokens"], dx, s["m"], s["v"], scale=SCALE, step=2, lr=1e-2)
    return [y, loss, dlogits, dlogits2, dx, dg, db, grad]


def _static(seed, n=700, rows=1500, dim=64, vocab=2050):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"table": r(rows, dim), "tokens": torch.randint(-1, 60, (n,), generator=g, device=DEV), "g": r(dim),
         "b": r(dim), "head": r(dim, vocab).bfloat16(), "teacher": r(n, 9), "w": r(n).abs(),
         "ids": torch.randint(0, vocab, (n, 9), generator=g, device=DEV), "p": r(rows, dim), "m": r(rows, dim),
         "v": r(rows, dim).abs()}
    s["head_t"] = s["head"].t().contiguous()
    return s


def test_captured_calls_replay_like_eager_ones():
    """Two graphs of the same calls, replayed in turn on new inputs with eager work between."""
    graphs = []
    for seed in (1, 2):
        s = _static(seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _calls(s)  # library handles of the two products
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _calls(s)
        graphs.append((g, s, out))
    for turn in range(3):
        for k, (g, s, out) in enumerate(graphs):
            new = _static(10 + 2 * turn + k)
            for name in s:
                s[name].copy_(new[name])
            g.replay()
            want = _calls(new)
            torch.cuda.synchronize()
            for a, b in zip(out + [s["p"], s["m"], s["v"]], want + [new["p"], new["m"], new["v"]]):
                assert torch.equal(a, b)


def test_captured_backward_pass_replays():
    """loss.backward() through the autograd functions, captured: the parameters' gradients are
    the graph's own buffers (no eager graph of these leaves exists)."""
    p, batch = _leaves(_model(4)), _batch(4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _loss(p, batch).backward()
        for t in p.values():
            t.grad = None
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _loss(p, batch).backward()
    for seed in (5, 6, 7):
        for a, b in zip(batch, _batch(seed)):
            a.copy_(b)
        g.replay()
        fresh = {k: t.detach().clone().requires_grad_(True) for k, t in p.items()}
        _loss(fresh, _batch(seed)).backward()
        torch.cuda.synchronize()
        for k in p:
            assert torch.equal(p[k].grad, fresh[k].grad), k


def test_calls_on_another_stream():
    s, t = _static(3), _static(3)
    side = torch.cuda.Stream()
    want = _calls(t)
    side.wait_stream(torch.cuda.current_stream())
    x = ma.embedding_forward(s["table"], s["tokens"], scale=SCALE, out_dtype=torch.bfloat16, stream=side)
    y, mean, rstd = ma.layer_norm_forward(x, s["g"], s["b"], stream=side)
    with torch.cuda.stream(side):
        logits = y @ s["head"]
    loss, dlogits = ma.distill_loss_grad(logits, s["teacher"], s["ids"], s["w"], temperature=TAU, stream=side)
    with torch.cuda.stream(side):
        dy = dlogits @ s["head_t"]
    dx, dg, db = ma.layer_norm_backward(dy, x, mean, rstd, s["g"], stream=side)
    grad = ma.embedding_backward(dx, s["tokens"], s["table"].shape[0], scale=SCALE, stream=side)
    ma.adamw_step_embedding(s["p"], s["tokens"], dx, s["m"], s["v"], scale=SCALE, step=2, lr=1e-2, stream=side)
    torch.cuda.synchronize()
    for a, b in zip([y, loss, dlogits, dx, dg, db, grad, s["p"], s["m"], s["v"]],
                    [want[i] for i in (0, 1, 2, 4, 5, 6, 7)] + [t["p"], t["m"], t["v"]]):
        assert torch.equal(a, b)


def test_inputs_dropped_while_another_stream_uses_them():
    """The caller's tensors are recorded on the stream that the work is given to: dropped right
    after the call, their memory is not handed out before that stream is done."""
    side = torch.cuda.Stream()
    n, dim, rows = 4096, 2048, 5000
    table = torch.randn(rows, dim, device=DEV)
    want = []
    for seed in range(3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        t = torch.randint(0, rows, (n,), generator=g, device=DEV)
        want.append((ma.embedding_backward(torch.randn(n, dim, generator=g, device=DEV), t, rows), table[t]))
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            busy = torch.tanh(busy @ busy)
    for seed in range(3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        t = torch.randint(0, rows, (n,), generator=g, device=DEV)
        dout = torch.randn(n, dim, generator=g, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        got.append((ma.embedding_backward(dout, t, rows, stream=side), ma.embedding_forward(table, t, stream=side)))
        del t, dout
        torch.full((n, dim), 1e30, device=DEV), torch.full((n,), rows - 1, device=DEV)  # the same sizes again
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_threads_at_once():
    """Calls from two threads on their own streams, workspaces allocated per call."""
    inputs, want = [_static(20), _static(21)], []
    for seed in (20, 21):
        t = _static(seed)
        want.append(_calls(t) + [t["p"], t["m"], t["v"]])
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = _calls(inputs[i])
                torch.cuda.current_stream().synchronize()
                got[i] = out + [inputs[i][k] for k in "pmv"]
        except Exception as e:  # pragma: no cover
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_single_rows_and_tokens():
    """Vectors and zero-dimensional tokens are batches of one."""
    v, table = torch.randn(64, device=DEV), torch.randn(50, 64, device=DEV)
    y, mean, rstd = ma.layer_norm_forward(v)
    rows = ma.layer_norm_forward(v[None])
    assert y.shape == (64,) and mean.shape == rstd.shape == () and torch.equal(y, rows[0][0])
    dx, dw, _ = ma.layer_norm_backward(y, v, mean, rstd)
    assert dx.shape == dw.shape == (64,)
    t = torch.tensor(3, device=DEV)
    assert torch.equal(ma.embedding_forward(table, t), table[3])
    grad = ma.embedding_backward(v, t, 50)
    assert torch.equal(grad[3], v) and not grad[:3].any() and not grad[4:].any()
    ids, one = torch.tensor([1, 5], device=DEV), torch.tensor(1.0, device=DEV)
    loss, dz = ma.distill_loss_grad(v, table[0, :2].contiguous(), ids, one)
    rows = ma.distill_loss_grad(v[None], table[:1, :2].contiguous(), ids[None], one[None])
    assert loss.shape == () and torch.equal(loss, rows[0][0]) and torch.equal(dz, rows[1][0])


def test_binding_checks_shapes():
    x = torch.zeros(6, 8, device=DEV)
    i = torch.zeros(6, dtype=torch.int64, device=DEV)
    f = torch.zeros(6, device=DEV)
    for bad in (lambda: ma.embedding_forward(x, i.float()), lambda: ma.embedding_forward(x.double(), i),
                lambda: ma.embedding_forward(x, i, out=x[:, :4]), lambda: ma.embedding_forward(f, i),
                lambda: ma.embedding_forward(x, i, out_dtype=torch.float64),
                lambda: ma.embedding_backward(x[:5], i, 9), lambda: ma.embedding_backward(x, i.cpu(), 9),
                lambda: ma.embedding_backward(x.t(), torch.zeros(8, dtype=torch.int64, device=DEV), 9),
                lambda: ma.embedding_backward(x[:1].expand(6, 8), i, 9),
                lambda: ma.embedding_backward(x, i, 9, grad=x),
                lambda: ma.adamw_step_embedding(x, i, x.clone(), x[:5], x, step=1, lr=1.0),
                lambda: ma.layer_norm_forward(x, f), lambda: ma.layer_norm_forward(x.double()),
                lambda: ma.layer_norm_forward(x, out=x.bfloat16()),
                lambda: ma.layer_norm_backward(x, x, f[:3], f), lambda: ma.layer_norm_backward(x.half(), x, f, f),
                lambda: ma.layer_norm_backward(x, x.clone(), f, f.clone(), accumulate=True),
                lambda: ma.layer_norm_backward(x, x, f, f, weight_grad=False, dweight=f),
                lambda: ma.distill_forward(x, x, i[:, None]), lambda: ma.distill_forward(x, x[:, :2], i.view(6, 1)),
                lambda: ma.distill_loss_grad(x, f[:, None], i[:, None], f[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ma.MuonAdamWError):
        ma.embedding_forward(x, i, out=x)  # over its own table
    with pytest.raises(ma.MuonAdamWError):
        ma.layer_norm_forward(x, out=x)
    with pytest.raises(ma.MuonAdamWError):
        ma.distill_forward(x, f[:, None], i[:, None], temperature=0.0)


def _every_call(s, x, stats, mean, stream):
    """Each entry point once, on tensors that are all there."""
    w, rows = s["w"], s["table"].shape[0]
    out = [ma.embedding_forward(s["table"], s["tokens"], scale=SCALE, stream=stream),
           *ma.layer_norm_forward(x, s["g"], s["b"], stream=stream),
           *ma.layer_norm_backward(x, x, mean, w, s["g"], stream=stream),
           ma.embedding_backward(x, s["tokens"], rows, stream=stream),
           *ma.distill_forward(x, s["teacher"], s["ids"], stream=stream),
           ma.distill_backward(x, s["teacher"], s["ids"], stats, w, stream=stream),
           *ma.distill_loss_grad(x, s["teacher"], s["ids"], w, stream=stream)]
    ma.adamw_step_embedding(s["p"], s["tokens"], x, s["m"], s["v"], step=1, lr=1e-2, stream=stream)
    return out + [s["p"].clone(), s["m"].clone(), s["v"].clone()] if stream is None else out


def _ready(seed):
    s = _static(seed, vocab=64)
    x = torch.randn(s["tokens"].numel(), 64, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    stats = torch.stack([x.amax(1), torch.exp(x - x.amax(1, keepdim=True)).sum(1)], 1)
    mean = x.mean(1)
    torch.cuda.synchronize()
    return s, x, stats, mean


def test_outputs_and_workspaces_are_the_streams_own_memory(monkeypatch):
    """What calls on the current stream have dropped is not handed to calls on another stream,
    which do not wait for the current one."""
    from adamw_optimizer_step_muon_amd import ops

    s, *rest = _ready(5)
    seen, call = [], ops._call
    monkeypatch.setattr(ops, "_call", lambda name, device, stream, *args: (
        seen.append((stream, {a for a in args if isinstance(a, int) and a > 1 << 32})),
        call(name, device, stream, *args)))
    inputs = {t.data_ptr() for t in [*s.values(), *rest]}
    for stream in (None, torch.cuda.Stream()):
        out = _every_call(s, *rest, stream)
        torch.cuda.synchronize()
        del out
    here, there = ({a for st, args in seen for a in args if (st is None) == k} - inputs for k in (True, False))
    assert len(seen) == 16 and len(here) > 10 and len(there) > 10
    assert not here & there


def test_a_call_beside_one_that_has_just_returned():
    """Calls of the same sizes on the current stream and, without a wait between them, on
    another: each has its own memory, and gives what it gives alone."""
    first, second = _ready(6), _ready(7)
    want = _every_call(*_ready(6), None), _every_call(*_ready(7), None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(2048, 2048, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        big = torch.tanh(big @ big)  # the current stream has work to come first
    a = _every_call(*first, None)
    b = _every_call(*second, side)
    torch.cuda.synchronize()
    b += [second[0][k] for k in "pmv"]
    for got, ref in ((a, want[0]), (b, want[1])):
        assert len(got) == len(ref)
        for p, q in zip(got, ref):
            assert torch.equal(p, q)


def test_writes_into_the_callers_tensors_advance_their_versions():
    """As torch's own in-place operations do, so that what autograd or the optimizer keeps of
    such a tensor is not taken for unchanged."""
    s, x, stats, mean = _ready(8)
    rows, w = s["table"].shape[0], s["w"]
    calls = {
        "lookup": lambda t: ma.embedding_forward(s["table"], s["tokens"], out=t[0]),
        "gradient": lambda t: ma.embedding_backward(x, s["tokens"], rows, grad=t[1]),
        "added": lambda t: ma.embedding_backward(x, s["tokens"], rows, grad=t[1], accumulate=True),
        "norm": lambda t: ma.layer_norm_forward(x, out=t[0]),
        "gain": lambda t: ma.layer_norm_backward(x, x, mean, w, dweight=t[2], bias_grad=False),
        "bias": lambda t: ma.layer_norm_backward(x, x, mean, w, dbias=t[2], weight_grad=False),
        "distilled": lambda t: ma.distill_backward(x, s["teacher"], s["ids"], stats, w, dlogits=t[0]),
        "both": lambda t: ma.distill_loss_grad(x, s["teacher"], s["ids"], w, dlogits=t[0])}
    written = {"lookup": 0, "gradient": 1, "added": 1, "norm": 0, "gain": 2, "bias": 2, "distilled": 0, "both": 0}
    for name, call in calls.items():
        t = [torch.zeros_like(x), torch.zeros_like(s["p"]), torch.zeros(64, device=DEV)]
        kept = [*t, x, stats, mean, *s.values()]
        before = [k._version for k in kept]
        call(t)
        assert [k._version > b for k, b in zip(kept, before)] == [i == written[name] for i in range(len(kept))], name
    state = [s["p"], s["m"], s["v"]]
    before = [k._version for k in state]
    ma.adamw_step_embedding(s["p"], s["tokens"], x, s["m"], s["v"], step=1, lr=1e-2)
    assert all(k._version > b for k, b in zip(state, before))

    # logits that a loss has kept for its backward pass
    z = x.clone().requires_grad_(True)
    logits = z * 1.0
    loss = ma.distill_loss(logits, s["teacher"], s["ids"]).sum()
    ma.distill_loss_grad(logits.detach(), s["teacher"], s["ids"], w, dlogits=logits.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # output gradients that the optimizer has kept
    table = torch.nn.Parameter(s["table"].clone())
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [table]}])
    dout = x.clone()
    opt.add_token_gradient(table, s["tokens"], dout)
    ma.layer_norm_forward(x, out=dout)
    with pytest.raises(RuntimeError, match="modified before step"):
        opt.step()
    # tensors without a version
    with torch.inference_mode():
        u = torch.empty_like(x)
    assert ma.layer_norm_forward(x, out=u)[0] is u


def test_tokens_and_teacher_lists_of_any_strides():
    """Slices of a batch's tokens and of longer teacher lists give what their copies give,
    on the current stream, on another, and through autograd."""
    g = torch.Generator(device=DEV).manual_seed(9)
    table = torch.randn(V, D, generator=g, device=DEV)
    tokens = torch.randint(-1, V, (6, 90), generator=g, device=DEV)[:, :-1]
    dout = torch.randn(6, 89, D, generator=g, device=DEV)
    logits = torch.randn(6, 89, V, generator=g, device=DEV)
    teacher = torch.randn(6, 89, 2 * K, generator=g, device=DEV)[..., :K]
    ids = torch.randint(-1, V, (K, 89, 6), generator=g, device=DEV).permute(2, 1, 0)
    w = torch.rand(6, 89, generator=g, device=DEV)
    assert not tokens.is_contiguous() and not teacher.is_contiguous() and not ids.is_contiguous()
    torch.cuda.synchronize()

    def run(tokens, teacher, ids, stream):
        p, m, v = table.clone(), torch.zeros_like(table), torch.zeros_like(table)
        torch.cuda.synchronize()
        loss, stats = ma.distill_forward(logits, teacher, ids, stream=stream)
        if stream is not None:
            stream.synchronize()
        ma.adamw_step_embedding(p, tokens, dout, m, v, step=1, lr=1e-2, stream=stream)
        out = [ma.embedding_forward(table, tokens, stream=stream), ma.embedding_backward(dout, tokens, V, stream=stream),
               loss, ma.distill_backward(logits, teacher, ids, stats, w, stream=stream),
               *ma.distill_loss_grad(logits, teacher, ids, w, stream=stream), p, m, v]
        torch.cuda.synchronize()
        a, b = table.clone().requires_grad_(True), logits.clone().requires_grad_(True)
        (ma.embedding(tokens, a) * dout).sum().backward()
        (ma.distill_loss(b, teacher, ids) * w).sum().backward()
        return out + [a.grad, b.grad]

    want = run(tokens.contiguous(), teacher.contiguous(), ids.contiguous(), None)
    for stream in (None, torch.cuda.Stream()):
        for a, b in zip(run(tokens, teacher, ids, stream), want):
            assert torch.equal(a, b)


def _two_groups(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    gain, table = torch.randn(D, generator=g, device=DEV), torch.randn(V, D, generator=g, device=DEV)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [gain], "lr": 1e-2}, {"kind": "adamw", "params": [table], "lr": 1e-2}])
    gain.grad = torch.randn(D, generator=g, device=DEV)
    pairs = [(torch.randint(0, V, (9,), generator=g, device=DEV), torch.randn(9, D, generator=g, device=DEV))
             for _ in range(2)]
    for tokens, dout in pairs:
        opt.add_token_gradient(table, tokens, dout)
    return opt, gain, table, pairs


def test_a_step_repeated_after_a_refusal_counts_everything_once(monkeypatch):
    """A step that fails, while it checks or while it adds up, and is called again."""
    from adamw_optimizer_step_muon_amd import ops

    opt, gain, table, pairs = _two_groups(1)
    want = _two_groups(1)
    dense = torch.randn(D, V, device=DEV).t()
    want[2].grad = dense.contiguous()
    want[0].step()
    table.grad = dense  # refused: not contiguous
    kept = [t.clone() for t in (gain, table)]
    with pytest.raises(ValueError, match="contiguous"):
        opt.step()
    assert torch.equal(gain, kept[0]) and torch.equal(table, kept[1])
    assert [g["step"] for g in opt.param_groups] == [0, 0]
    table.grad = dense.contiguous()
    opt.step()
    for a, b in zip((gain, table, table.grad), (want[1], want[2], want[2].grad)):
        assert torch.equal(a, b)

    # the second of two additions fails once
    opt, gain, table, pairs = _two_groups(2)
    backward, calls = ops.embedding_backward, []

    def fails_once(*args, **kw):
        calls.append(1)
        if len(calls) == 2:
            raise MemoryError
        return backward(*args, **kw)

    monkeypatch.setattr(ops, "embedding_backward", fails_once)
    gain.grad = None
    with pytest.raises(MemoryError):
        opt.step()
    opt.step()
    monkeypatch.undo()
    ref = backward(pairs[0][1], pairs[0][0], V)
    backward(pairs[1][1], pairs[1][0], V, grad=ref, accumulate=True)
    assert torch.equal(table.grad, ref) and opt.param_groups[1]["step"] == 1


@pytest.mark.parametrize("additions", [1, 2])
def test_a_step_waits_for_the_stream_that_made_a_token_gradient(additions):
    """Output gradients that another stream is still computing when step() is called."""
    g = torch.Generator(device=DEV).manual_seed(3)
    rows, dim, n = 3000, 512, 2048
    values, a = torch.randn(rows, dim, generator=g, device=DEV), torch.randn(n, dim, generator=g, device=DEV)
    turn = torch.randn(dim, dim, generator=g, device=DEV) / dim ** 0.5
    tokens = torch.randint(0, rows, (n,), generator=g, device=DEV)

    def made():
        x = a
        for _ in range(200):
            x = torch.tanh(x @ turn)
        return x

    def run(stream):
        table = values.clone()
        opt = ma.MuonAdamW([{"kind": "adamw", "params": [table], "lr": 1e-2}])
        torch.cuda.synchronize()
        for _ in range(additions):
            with torch.cuda.stream(stream):
                opt.add_token_gradient(table, tokens, made())
        opt.step()
        torch.cuda.synchronize()
        return table

    want = run(torch.cuda.current_stream())
    assert torch.equal(run(torch.cuda.Stream()), want)


def test_a_captured_step_on_tokens_replays():
    """Forward, backward and step by token gradients in one graph, with the embedding's forward
    pass (so its backward) on another stream of the capture; every replay against eager steps."""
    p, batch = _leaves(_model(11)), _batch(11)
    start = {k: t.detach().clone() for k, t in p.items()}
    warm = _leaves(_model(11))
    o = _optimizer(warm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _loss(warm, _batch(11), o).backward()
        o.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    del warm, o
    opt = _optimizer(p)
    leaves = {k: p[k].data for k in p}
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            loss = _loss(p, batch, opt)
        loss.backward()  # on the forward pass's stream; torch orders this one behind its gradients
        opt.step()
        del loss
        here.wait_stream(other)
    assert p["table"].grad is None
    q = _leaves(_model(11))
    eager = _optimizer(q)
    for seed in (12, 13, 14):
        for a, b in zip(batch, _batch(seed)):
            a.copy_(b)
        graph.replay()
        for g in eager.param_groups:
            g["step"] = 0  # the captured step's count
        _loss(q, _batch(seed), eager).backward()
        eager.step()
        eager.zero_grad()
        torch.cuda.synchronize()
        for k in p:
            assert torch.equal(leaves[k], q[k].data), k
    assert not torch.equal(leaves["table"], start["table"])


def test_a_backward_pass_and_a_step_captured_apart():
    """Output gradients made in one graph and stepped by another, on their own streams; the
    replays follow each other on one stream."""
    table = torch.randn(V, D, device=DEV)
    tokens, a = torch.randint(0, V, (30,), device=DEV), torch.randn(30, D, device=DEV)
    opt = ma.MuonAdamW([{"kind": "adamw", "params": [table], "lr": 1e-2}])
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first, stream=torch.cuda.Stream()):
        opt.add_token_gradient(table, tokens, torch.tanh(a))
    with torch.cuda.graph(second, stream=torch.cuda.Stream()):
        opt.step()
    q = [table.clone(), torch.zeros_like(table), torch.zeros_like(table)]
    for _ in range(3):
        a.add_(0.5)
        first.replay()
        second.replay()
        ma.adamw_step_embedding(q[0], tokens, torch.tanh(a), q[1], q[2], step=1, lr=1e-2)
        torch.cuda.synchronize()
        assert torch.equal(table, q[0])


def test_binding_refuses_outputs_that_are_no_tensors():
    x, i = torch.zeros(6, 8, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV)
    f, a = torch.zeros(6, device=DEV), torch.zeros(6, 1, device=DEV)
    for call in (lambda: ma.embedding_forward(x, i, out=[1.0]), lambda: ma.layer_norm_forward(x, out=3),
                 lambda: ma.distill_loss_grad(x, a, i[:, None], f, dlogits="x")):
        with pytest.raises(TypeError, match="torch.Tensor"):
            call()
    with pytest.raises(ValueError, match="dimension"):
        ma.embedding_backward(f[0], i[0], 10)
