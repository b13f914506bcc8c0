"""The operators together, as a recurrent language model runs them: token
embedding -> LSTM -> gated delta rule -> logits -> log-probabilities, trained
one step and then decoded token by token.  The projections between them and the
64-bit model are torch's; gradients are compared with its autograd.

Tolerance: the LSTM's own (1e-4 of the largest value in fp32); what follows it
adds float roundings only."""
import pytest
import torch

from backward_lstm_fwd_b200 import binding as L
from backward_lstm_fwd_b200 import build as lbuild

pytestmark = pytest.mark.gpu
T, B, VOCAB, I, H, HK, HV, K, V = 70, 3, 53, 24, 32, 2, 4, 16, 8
SCALE, TEMPERATURE = 2.0, 0.9


@pytest.fixture(scope="module", autouse=True)
def _built():
    lbuild.build()


def parameters():
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return {"table": rn(VOCAB, I), "W": 0.3 * rn(4 * H, H + I), "b": 0.1 * rn(4 * H),
            "qkv": 0.5 * rn(H, 2 * HK * K + HV * V), "gates": 0.5 * rn(H, 2 * HV), "out": 0.5 * rn(HV * V, VOCAB)}


def project(p, y):
    """q, k, v, log decay and beta of the delta rule from the LSTM's outputs."""
    t, b = y.shape[:2]
    q, k, v = (y @ p["qkv"]).split([HK * K, HK * K, HV * V], dim=-1)
    unit = torch.nn.functional.normalize
    g, beta = (y @ p["gates"]).split(HV, dim=-1)
    return (unit(q.view(t, b, HK, K), dim=-1), unit(k.view(t, b, HK, K), dim=-1), v.reshape(t, b, HV, V),
            -torch.nn.functional.softplus(g), torch.sigmoid(beta))


def model64(p, ids, targets):
    """Log-probability of every target and every row's entropy, in float64."""
    p = {n: t.double().detach().requires_grad_() for n, t in p.items()}
    x = SCALE * torch.where((ids >= 0)[..., None], p["table"][ids.clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda"))
    h = c = torch.zeros(B, H, dtype=torch.float64, device="cuda")
    ys = []
    for t in range(ids.shape[0]):
        i, f, g, o = (torch.cat([h, x[t]], -1) @ p["W"].t() + p["b"]).chunk(4, -1)
        c = torch.sigmoid(f) * c + torch.sigmoid(i) * torch.tanh(g)
        h = torch.sigmoid(o) * torch.tanh(c)
        ys.append(h)
    q, k, v, g, beta = project(p, torch.stack(ys))
    q, k = (s.repeat_interleave(HV // HK, dim=2) for s in (q, k))
    S, os = torch.zeros(B, HV, K, V, dtype=torch.float64, device="cuda"), []
    for t in range(ids.shape[0]):
        S = torch.exp(g[t])[..., None, None] * S
        u = beta[t][..., None] * (v[t] - (k[t][..., None] * S).sum(2))
        S = S + k[t][..., None] * u[:, :, None]
        os.append(K ** -0.5 * (q[t][..., None] * S).sum(2))
    logits = torch.stack(os).reshape(-1, HV * V) @ p["out"]
    lp = torch.log_softmax(logits / TEMPERATURE, 1)
    return p, logits, lp.gather(1, targets.reshape(-1, 1))[:, 0], -(lp.exp() * lp).sum(1)


def close(name, got, ref, tol=2e-4):
    ref = ref.detach()
    err = float((got.detach().double() - ref).abs().max() / ref.abs().max())
    assert err <= tol, (name, err)


def test_training_step_and_decoding():
    p = parameters()
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, VOCAB, (T, B), generator=g, device="cuda")
    ids[3, 1] = -1
    targets = torch.randint(0, VOCAB, (T, B), generator=g, device="cuda")
    weight = torch.rand(T * B, generator=g, device="cuda")

    x = L.embed(ids, p["table"], SCALE)
    ls = L.forward(x, p["W"], p["b"])
    y = ls.y.detach().requires_grad_()
    leaves = {n: p[n].detach().requires_grad_() for n in ("qkv", "gates")}
    five = project(leaves, y)
    gs = L.gdr_forward(*(t.detach().contiguous() for t in five), save=True)
    flat = gs.o.reshape(T * B, HV * V)
    logits = flat @ p["out"]
    lp = L.logprobs(logits, targets.reshape(-1), top=3, temperature=TEMPERATURE)

    q, logits64, logp64, entropy64 = model64(p, ids, targets)
    close("logp", lp.logp, logp64)
    close("entropy", lp.entropy, entropy64)
    assert torch.equal(lp.top_ids.long(), torch.argsort(-logits, dim=1, stable=True)[:, :3])

    # loss = -sum weight logp - 0.1 sum entropy
    dlogits = L.logprobs_backward(lp, logits, targets.reshape(-1), dlogp=-weight, dentropy=torch.full_like(weight, -0.1),
                                  temperature=TEMPERATURE)
    dout = (dlogits @ p["out"].t()).view(T, B, HV, V)
    gg = L.gdr_backward(gs, *(t.detach().contiguous() for t in five), dout=dout)
    torch.autograd.backward(five, [gg.dq, gg.dk, gg.dv, gg.dg, gg.dbeta])
    lg = L.backward(ls, x, p["W"], dy=y.grad)
    got = {"table": L.embed_backward(ids, lg.dx, VOCAB, SCALE), "W": lg.dW, "b": lg.db, "qkv": leaves["qkv"].grad,
           "gates": leaves["gates"].grad, "out": flat.t() @ dlogits}
    (-(weight.double() * logp64).sum() - 0.1 * entropy64.sum()).backward()
    for n, t in got.items():
        close("d" + n, t, q[n].grad, 1e-3)

    # the last tokens again, one at a time, from the states after the others
    split = T - 4
    ls = L.forward(x[:split].contiguous(), p["W"], p["b"])
    gs = L.gdr_forward(*(t.detach().contiguous() for t in project(p, ls.y)))
    h, c, S = ls.hT, ls.cT, gs.sT
    for t in range(split, T):
        ls = L.forward(L.embed(ids[t:t + 1], p["table"], SCALE), p["W"], p["b"], h0=h, c0=c)
        h, c = ls.hT, ls.cT
        gs = L.gdr_forward(*(s.detach().contiguous() for s in project(p, ls.y)), s0=S, sT=S)
        one = L.logprobs(gs.o.reshape(B, HV * V) @ p["out"], targets[t], top=2, temperature=TEMPERATURE)
        close(f"step {t}", one.logp, logp64.view(T, B)[t])


def test_stream_argument():
    """A call on a stream that is not the current one works and allocates there."""
    p = parameters()
    ids = torch.arange(T * B, device="cuda").view(T, B) % VOCAB
    x = L.embed(ids, p["table"], SCALE)
    dx = torch.randn_like(x)
    five = [t.contiguous() for t in project({n: p[n] for n in p}, torch.randn(T, B, H, device="cuda"))]
    logits = torch.randn(T * B, VOCAB, device="cuda")
    t = ids.reshape(-1)

    def run(**kw):
        gs = L.gdr_forward(*five, save=True, **kw)
        gr = L.gdr_backward(gs, *five, dout=gs.o, **kw)
        few = L.gdr_forward(*(f[:3] for f in five), **kw)
        lp = L.logprobs(logits, t, top=2, **kw)
        d = L.logprobs_backward(lp, logits, t, dlogp=lp.entropy, **kw)
        return (L.embed(ids, p["table"], SCALE, **kw), L.embed_backward(ids, dx, VOCAB, **kw), gs.o, gr.dk, gr.dg, few.o,
                lp.logp, d)

    want = run()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        torch.cuda.synchronize()
        got = run(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_inputs_let_go_while_another_stream_works():
    """Temporaries given to a call on another stream, and a state used on another stream than it was made on: their memory
    is not handed out again before the call is done."""
    p = parameters()
    ids = torch.arange(T * B, device="cuda").view(T, B) % VOCAB
    t = torch.arange(300, device="cuda")
    logits = torch.randn(300, 2111, device="cuda")
    five = [f.contiguous().repeat(4, 5, *[1] * (f.dim() - 2)) for f in project(p, torch.randn(T, B, H, device="cuda"))]
    lp = L.logprobs(logits, t)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    for call, inputs in (
            (lambda i, w, **kw: [L.embed(i, w, **kw)], [ids, torch.randn(VOCAB, 20000, device="cuda")]),
            (lambda i, d, **kw: [L.embed_backward(i, d, VOCAB, **kw)], [ids, torch.randn(T, B, 3000, device="cuda")]),
            (lambda x, t, **kw: [L.logprobs(x, t, **kw).logp], [logits, t]),
            (lambda x, t, g, **kw: [L.logprobs_backward(lp, x, t, dlogp=g, **kw)], [logits, t, torch.rand(300, device="cuda")]),
            (lambda *f, **kw: [L.gdr_forward(*f, **kw).o], five),
            (lambda *f, **kw: [L.gdr_forward(*(x[:5] for x in f), **kw).o], five)):
        want = call(*inputs)
        given = [x.clone() for x in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # (some 50 ms)
        got = call(*given, stream=side)
        del given
        again = [torch.ones_like(x) for x in inputs]  # would take the places of what was let go
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del again
    # states
    st = L.gdr_forward(*five, save=True)
    want, wd = L.gdr_backward(st, *five, dout=st.o), L.logprobs_backward(lp, logits, t, dlogp=lp.entropy)
    with torch.cuda.stream(side):
        side.wait_stream(here)
        st, lp = L.gdr_forward(*five, save=True), L.logprobs(logits, t)
        dout, dl = st.o.clone(), lp.entropy.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got, gd = L.gdr_backward(st, *five, dout=dout), L.logprobs_backward(lp, logits, t, dlogp=dl)
    sizes = [x.numel() * x.element_size() for x in (st.states, st.deltas, st.ws, lp._buf)]
    del st, lp
    with torch.cuda.stream(side):
        again = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert torch.equal(gd, wd)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(getattr(got, n), getattr(want, n)), n
    del again


def test_other_streams_inside_a_graph():
    """Calls on a stream forked from a captured one, their inputs' memory known to the allocator there too."""
    ids = torch.arange(T * B, device="cuda").view(T, B) % VOCAB
    table, dx, logits = torch.randn(VOCAB, I, device="cuda"), torch.randn(T, B, I, device="cuda"), torch.randn(T * B, VOCAB, device="cuda")
    five = [t.contiguous() for t in project(parameters(), torch.randn(T, B, H, device="cuda"))]

    def run(**kw):
        gs = L.gdr_forward(*(f + 0 for f in five), save=True, **kw)
        lp = L.logprobs(logits, ids.reshape(-1), **kw)
        return [L.embed(ids, table, **kw), L.embed_backward(ids, dx, VOCAB, **kw), gs.o, L.gdr_backward(gs, *five, dout=gs.o, **kw).dk,
                lp.logp, L.logprobs_backward(lp, logits, ids.reshape(-1), dlogp=lp.entropy, **kw)]

    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
