"""lstm_gdr_fwd / lstm_gdr_bwd against the recurrence itself in 64 bits (token
by token, gradients by torch's autograd of it).

Tolerance.  The kernels compute as floats do: a value goes through sums of
K + 64 + 64 products a chunk (forward; the same again backward, and once more
for the gradients of q, k, g and beta), each addition rounding by 2^-24 of
the sums' magnitude at most.  Over `chunks` chunks that is
384 * chunks * 2^-24 of the largest value for forward results, three times
that for gradients, plus the rounding to the output's type."""
import pytest
import torch

from backward_lstm_fwd_b200 import binding as L
from backward_lstm_fwd_b200 import build as lbuild

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    lbuild.build()


def make(T, B, Hk, Hv, K, V, dt, seed=0, s0=True):
    gen = torch.Generator(device="cuda").manual_seed(seed + T + B + K)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = {"q": torch.nn.functional.normalize(rn(T, B, Hk, K), dim=-1).to(DT[dt]),
         "k": torch.nn.functional.normalize(rn(T, B, Hk, K), dim=-1).to(DT[dt]),
         "v": rn(T, B, Hv, V).to(DT[dt]),
         "g": -torch.nn.functional.softplus(rn(T, B, Hv) - 2), "beta": torch.sigmoid(rn(T, B, Hv)),
         "s0": 0.3 * rn(B, Hv, K, V) if s0 else None}
    return x, rn(T, B, Hv, V).to(DT[dt]), rn(B, Hv, K, V)


def reference(q, k, v, g, beta, s0, lengths, scale):
    """The recurrence in float64 (differentiable in its inputs)."""
    T, B, Hk, K = q.shape
    Hv, V = v.shape[2:]
    q, k = (t.repeat_interleave(Hv // Hk, dim=2) for t in (q, k))
    S = s0 if s0 is not None else torch.zeros(B, Hv, K, V, dtype=torch.float64, device=q.device)
    out = []
    for t in range(T):
        Sd = torch.exp(g[t])[..., None, None] * S
        x = v[t] - (k[t][..., None] * Sd).sum(2)
        Sn = Sd + k[t][..., None] * (beta[t][..., None] * x)[:, :, None]
        o = scale * (q[t][..., None] * Sn).sum(2)
        if lengths is not None:
            real = (t < lengths)[:, None, None]
            o = torch.where(real, o, torch.zeros_like(o))
            Sn = torch.where(real[..., None], Sn, S)
        S = Sn
        out.append(o)
    return (torch.stack(out) if out else v), S


def close(name, got, ref, chunks, times=1):
    assert got.shape == ref.shape, name
    if not ref.numel():
        return
    assert bool(torch.isfinite(got).all()), name
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    tol = half * ref.abs() + times * 384 * chunks * 2.0 ** -24 * ref.abs().max() + tiny
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{name}: {float((err / tol).max()):.3g} of the tolerance"


def check(x, dout, dsT, lengths=None, scale=None, grads=True):
    T, B, Hk, K = x["q"].shape
    scale = K ** -0.5 if scale is None else scale
    chunks = max(1, -(-T // 64))
    names = [n for n in ("q", "k", "v", "g", "beta", "s0") if x[n] is not None]
    d = {n: x[n].double().requires_grad_(grads) if x[n] is not None else None for n in x}
    o, S = reference(**d, lengths=lengths, scale=scale)
    st = L.gdr_forward(**x, lengths=lengths, scale=scale, save=grads)
    close("o", st.o, o.detach(), chunks)
    close("sT", st.sT, S.detach(), chunks)
    if not grads:
        return st
    gr = L.gdr_backward(st, x["q"], x["k"], x["v"], x["g"], x["beta"], dout=dout, dsT=dsT, lengths=lengths, scale=scale)
    loss = (o * dout.double()).sum() if dout is not None else 0
    loss = loss + ((S * dsT.double()).sum() if dsT is not None else 0)
    want = torch.autograd.grad(loss, [d[n] for n in names], allow_unused=True)
    for n, w in zip(names, want):
        w = torch.zeros_like(d[n]) if w is None else w
        close("d" + n, getattr(gr, "d" + n), w, chunks, 3)
    return st, gr


SHAPES = [(1, 1, 1, 1, 8, 8), (5, 2, 1, 2, 16, 24), (16, 3, 2, 2, 64, 128), (17, 1, 1, 1, 64, 64), (64, 2, 1, 1, 128, 128),
          (65, 1, 2, 4, 128, 64), (130, 2, 1, 3, 40, 72), (200, 1, 1, 1, 96, 256), (129, 1, 2, 2, 72, 136), (333, 2, 1, 2, 128, 128)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dt):
    x, _, _ = make(*shape, dt)
    check(x, None, None, grads=False)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, dt):
    check(*make(*shape, dt))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(70, 20, 2, 4, 16, 8), (65, 40, 1, 3, 72, 72), (40, 3, 1, 4, 128, 64)], ids=str)
def test_shared_key_heads(shape, dt):
    """Value heads of a group one after another in a block (many blocks), or a block each (few)."""
    check(*make(*shape, dt))


@pytest.mark.parametrize("dt", list(DT))
def test_lengths(dt):
    x, dout, dsT = make(150, 6, 1, 2, 64, 40, dt)
    lengths = torch.tensor([150, 0, 1, 64, 65, 149], dtype=torch.int32, device="cuda")
    st, gr = check(x, dout, dsT, lengths=lengths, scale=0.7)
    for b, n in enumerate(lengths.tolist()):
        for t in (st.o, gr.dq, gr.dk, gr.dv, gr.dg, gr.dbeta):
            assert not t[n:, b].any()
    assert torch.equal(st.sT[1], x["s0"][1]) and torch.equal(gr.ds0[1], dsT[1])
    clamped = torch.tensor([999, -5, 1, 64, 65, 149], dtype=torch.int32, device="cuda")
    assert torch.equal(L.gdr_forward(**x, lengths=clamped, scale=0.7, save=True).o, st.o)
    y = {n: t[:9].contiguous() if n != "s0" else t for n, t in x.items()}  # token by token
    check(y, None, None, lengths=torch.tensor([9, 0, 1, 8, 4, 2], dtype=torch.int32, device="cuda"), grads=False)


def test_optional_inputs():
    x, dout, dsT = make(70, 2, 1, 1, 32, 16, "bf16", s0=False)
    check(x, dout, dsT)
    check(x, dout, None)
    st, gr = check(x, None, dsT)
    x, dout, _ = make(70, 2, 1, 1, 32, 16, "bf16")
    check(x, None, None, grads=False)


def test_padding_values_do_not_matter():
    """NaN and infinities behind a sequence's length reach nothing."""
    x, dout, dsT = make(100, 2, 1, 1, 64, 64, "bf16")
    lengths = torch.tensor([70, 100], dtype=torch.int32, device="cuda")
    want = L.gdr_forward(**x, lengths=lengths, save=True)
    wg = L.gdr_backward(want, *(x[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT, lengths=lengths)
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "g", "beta"):
        y[n][70:, 0] = float("nan") if n != "v" else float("inf")
    dout = dout.clone()
    dout[70:, 0] = float("nan")
    got = L.gdr_forward(**y, lengths=lengths, save=True)
    gg = L.gdr_backward(got, *(y[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT, lengths=lengths)
    assert torch.equal(got.o, want.o) and torch.equal(got.sT, want.sT)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
        assert torch.equal(getattr(gg, n), getattr(wg, n)), n


@pytest.mark.parametrize("T", [9, 140])
def test_forgetting(T):
    """Strong decays keep their neighbours' digits; -inf forgets everything before it."""
    x, dout, dsT = make(T, 1, 1, 2, 32, 24, "fp32")
    x["g"][:, :, 0] = -30.0
    x["g"][::3, :, 0] = -0.01
    check(x, dout, dsT)
    x["g"][5, :, 1] = float("-inf")
    x["g"][T // 2, :, 1] = float("-inf")
    st = L.gdr_forward(**x, save=True)
    d = {n: t.double() for n, t in x.items()}
    o, S = reference(**d, lengths=None, scale=32 ** -0.5)
    close("o", st.o, o, -(-T // 64))
    close("sT", st.sT, S, -(-T // 64))
    gr = L.gdr_backward(st, *(x[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT)
    assert all(bool(torch.isfinite(getattr(gr, n)).all()) for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"))
    assert not gr.dg[5, :, 1].any()
    late = dout.clone()
    late[:5, :, 1] = 0  # nothing that saw s0 counts: token 5 forgets it
    gr = L.gdr_backward(st, *(x[n] for n in ("q", "k", "v", "g", "beta")), dout=late, dsT=dsT)
    assert not gr.ds0[:, 1].any() and gr.ds0[:, 0].any()


def test_beta_and_decay_limits():
    """beta 0 (nothing is written), beta 1 with g 0 (a pure delta rule), beta above 1."""
    x, dout, dsT = make(100, 1, 1, 3, 64, 32, "fp32")
    x["beta"][:, :, 0] = 0.0
    x["beta"][:, :, 1] = 1.0
    x["g"][:, :, 1] = 0.0
    x["beta"][:, :, 2] = 1.7
    check(x, dout, dsT)


def test_equal_keys():
    """One key for a whole chunk: the triangular system is as full as it gets."""
    x, dout, dsT = make(64, 1, 1, 1, 16, 16, "fp32")
    x["k"][:] = x["k"][:1]
    x["g"][:] = 0
    check(x, dout, dsT)


def test_slices_of_one_projection():
    T, B, Hk, Hv, K, V = 90, 3, 2, 4, 32, 24
    x, dout, dsT = make(T, B, Hk, Hv, K, V, "bf16")
    wide = torch.zeros(T, B, 2 * Hk * K + Hv * V + 8, dtype=torch.bfloat16, device="cuda")
    q = wide[..., : Hk * K].view(T, B, Hk, K)
    k = wide[..., Hk * K: 2 * Hk * K].view(T, B, Hk, K)
    v = wide[..., 2 * Hk * K: 2 * Hk * K + Hv * V].view(T, B, Hv, V)
    for a, n in ((q, "q"), (k, "k"), (v, "v")):
        a.copy_(x[n])
    want = L.gdr_forward(**x, save=True)
    got = L.gdr_forward(q, k, v, x["g"], x["beta"], x["s0"], save=True)
    assert torch.equal(got.o, want.o) and torch.equal(got.sT, want.sT)
    a = L.gdr_backward(want, x["q"], x["k"], x["v"], x["g"], x["beta"], dout=dout, dsT=dsT)
    b = L.gdr_backward(got, q, k, v, x["g"], x["beta"], dout=dout, dsT=dsT)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
        assert torch.equal(getattr(a, n), getattr(b, n))
    few = L.gdr_forward(q[:4], k[:4], v[:4], x["g"][:4], x["beta"][:4], x["s0"])
    assert torch.equal(few.o, L.gdr_forward(*(x[n][:4].contiguous() for n in ("q", "k", "v", "g", "beta")), x["s0"]).o)


def test_a_sequence_in_parts():
    """A prompt in chunks, then token by token with the state in place, is the whole sequence."""
    T, B, Hk, Hv, K, V = 150, 2, 1, 2, 64, 64
    x, _, _ = make(T, B, Hk, Hv, K, V, "bf16")
    whole = L.gdr_forward(**x)
    part = {n: x[n][:131] for n in ("q", "k", "v", "g", "beta")}
    st = L.gdr_forward(**part, s0=x["s0"])
    state, outs = st.sT, [st.o]
    for t in range(131, T):
        y = {n: x[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")}
        r = L.gdr_forward(**y, s0=state, sT=state)
        assert r.sT is state
        outs.append(r.o)
    ref, S = reference(**{n: t.double() for n, t in x.items()}, lengths=None, scale=K ** -0.5)
    close("o", torch.cat(outs), ref, 3)
    close("sT", state, S, 3)
    close("whole", whole.o, ref, 3)


@pytest.mark.parametrize("shape,dt", [((2050, 1, 1, 1, 128, 128), "bf16"), ((1500, 2, 1, 2, 64, 40), "fp16"),
                                      ((900, 1, 1, 2, 96, 256), "fp32"), ((256, 1, 1, 1, 32, 8), "bf16"),
                                      ((1100, 3, 1, 1, 128, 136), "fp16")], ids=str)
def test_long_with_few_heads(shape, dt):
    """Chunks in segments side by side, joined by their transition matrices."""
    x, dout, dsT = make(*shape, dt)
    d = L.gdr_dims(*shape, DT[dt])
    state = shape[1] * shape[3] * shape[4] * shape[5] * 4
    # (a split call keeps the starts of its segments)
    many = L.gdr_dims(shape[0], 64, *shape[2:3], 64 * shape[2], *shape[4:], DT[dt])
    per_chunk = lambda e, heads: L.gdr_fwd_workspace_size(e, True) / heads  # noqa: E731
    assert per_chunk(d, shape[1] * shape[3]) > per_chunk(many, 64 * 64 * shape[2]) + state / (shape[1] * shape[3])
    check(x, dout, dsT)
    lengths = torch.randint(0, shape[0] + 1, (shape[1],), dtype=torch.int32, device="cuda")
    lengths[0] = shape[0] * 2 // 3
    check(x, dout, dsT, lengths=lengths)
    x["s0"] = None
    check(x, dout, None)


def test_gradient_by_differences():
    """dg and dbeta against central differences of the 64-bit recurrence."""
    T, B, Hk, Hv, K, V = 80, 1, 1, 1, 16, 8
    x, dout, dsT = make(T, B, Hk, Hv, K, V, "fp32")
    st = L.gdr_forward(**x, save=True)
    gr = L.gdr_backward(st, *(x[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT)
    d = {n: t.double() for n, t in x.items()}

    def loss(y):
        o, S = reference(**y, lengths=None, scale=K ** -0.5)
        return float((o * dout.double()).sum() + (S * dsT.double()).sum())

    for n, got in (("g", gr.dg), ("beta", gr.dbeta)):
        for t in (0, 1, 40, 63, 64, 79):
            lo, hi = ({**d, n: d[n].clone()} for _ in range(2))
            lo[n][t] -= 1e-5
            hi[n][t] += 1e-5
            slope = (loss(hi) - loss(lo)) / 2e-5
            # differences: about 1e-10 of truncation and 1e-16 / 1e-5 of cancellation, of values near the largest gradient
            assert abs(slope - float(got[t])) <= 3 * 384 * 2 * 2.0 ** -24 * float(got.abs().max()) + 1e-6 * abs(slope) + 1e-7


def test_empty():
    e = dict(device="cuda")
    z = lambda *s: torch.zeros(*s, **e)  # noqa: E731
    s0 = torch.randn(2, 2, 8, 8, **e)
    st = L.gdr_forward(z(0, 2, 1, 8), z(0, 2, 1, 8), z(0, 2, 2, 8), z(0, 2, 2), z(0, 2, 2), s0)
    assert torch.equal(st.sT, s0) and st.o.shape == (0, 2, 2, 8)
    st = L.gdr_forward(z(0, 2, 1, 8), z(0, 2, 1, 8), z(0, 2, 2, 8), z(0, 2, 2), z(0, 2, 2), s0, save=True)
    gr = L.gdr_backward(st, z(0, 2, 1, 8), z(0, 2, 1, 8), z(0, 2, 2, 8), z(0, 2, 2), z(0, 2, 2), dsT=s0)
    assert torch.equal(gr.ds0, s0)
    L.gdr_forward(z(70, 0, 1, 8), z(70, 0, 1, 8), z(70, 0, 2, 8), z(70, 0, 2), z(70, 0, 2))


def test_streams_graphs_and_status():
    x, dout, dsT = make(100, 2, 1, 2, 64, 64, "bf16")
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want = L.gdr_forward(**x, save=True)
    wg = L.gdr_backward(want, *five, dout=dout, dsT=dsT)
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            st = L.gdr_forward(**x, save=True)
            outs.append((st, L.gdr_backward(st, *five, dout=dout, dsT=dsT)))
    torch.cuda.synchronize()
    for st, gr in outs:
        assert torch.equal(st.o, want.o) and torch.equal(gr.dk, wg.dk) and torch.equal(gr.dg, wg.dg)
    buf = {n: torch.zeros_like(t) for n, t in x.items()}
    ws = L.empty_workspace(L.gdr_bwd_workspace_size(want.dims), "cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = L.gdr_forward(**buf, save=True, ws=ws)
        gr = L.gdr_backward(st, *(buf[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT, ws=ws)
    for n in x:
        buf[n].copy_(x[n])
    g.replay()
    torch.cuda.synchronize()
    assert L.lstm_status(ws) == L.LSTM_OK
    assert torch.equal(st.o, want.o) and torch.equal(st.sT, want.sT)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
        assert torch.equal(getattr(gr, n), getattr(wg, n)), n


def test_step_in_one_graph():
    """Forward and backward captured together, the forward's workspace kept between them; replayed on new
    inputs, and the backward taken twice from one state."""
    x, dout, dsT = make(150, 2, 2, 4, 64, 72, "fp16")
    y, _, _ = make(150, 2, 2, 4, 64, 72, "fp16", seed=1)
    buf = {n: t.clone() for n, t in x.items()}
    names = ("q", "k", "v", "g", "beta")
    five = [buf[n] for n in names]
    L.gdr_forward(**buf, save=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = L.gdr_forward(**buf, save=True)
        once = L.gdr_backward(st, *five, dout=dout, dsT=dsT)
        again = L.gdr_backward(st, *five, dout=dout, dsT=dsT)
    for z in (y, x):
        for n in z:
            buf[n].copy_(z[n] if n != "beta" else z[n] * 0.5)
        graph.replay()
        torch.cuda.synchronize()
        ws = L.empty_workspace(L.gdr_bwd_workspace_size(st.dims), "cuda")
        own = L.gdr_forward(**{n: t.clone() for n, t in buf.items()}, save=True, ws=ws)  # keeps no workspace
        assert own.ws is None and st.ws is not None
        want = L.gdr_backward(own, *[t.clone() for t in five], dout=dout, dsT=dsT, ws=ws)
        assert torch.equal(st.o, own.o) and L.lstm_status(ws) == L.LSTM_OK
        for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
            assert torch.equal(getattr(once, n), getattr(want, n)) and torch.equal(getattr(again, n), getattr(want, n)), n


@pytest.mark.parametrize("T", [3, 100, 1500])
def test_state_in_place(T):
    """sT is s0, also where the sequence is split over blocks."""
    x, _, _ = make(T, 1, 1, 2, 64, 64, "bf16")
    want = L.gdr_forward(**x)
    for _ in range(3):
        state = x["s0"].clone()
        got = L.gdr_forward(*(x[n] for n in ("q", "k", "v", "g", "beta")), s0=state, sT=state)
        assert torch.equal(got.o, want.o) and torch.equal(state, want.sT)


def test_state_of_other_sizes():
    """A backward whose sizes are not its forward's would read past what the
    forward kept."""
    x, dout, dsT = make(100, 2, 2, 4, 64, 64, "bf16")
    st = L.gdr_forward(**x, save=True)
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    wide = [t.repeat(1, 1, 2, 1) for t in five[:2]]  # four key heads
    long = [torch.cat([t, t[..., :32]], -1).contiguous() for t in five[:2]]  # K = 96
    for q, k in (wide, long, [t.half() for t in five[:2]]):
        with pytest.raises(ValueError):
            L.gdr_backward(st, q, k, five[2].to(q.dtype), *five[3:], dout=dout.to(q.dtype), dsT=dsT if q.shape[-1] == 64 else None)
    with pytest.raises(ValueError, match="other sizes"):
        L.gdr_backward(st, *wide, *five[2:], dout=dout, dsT=dsT)
    with pytest.raises(ValueError, match="kept nothing"):
        L.gdr_backward(L.gdr_forward(**x), *five, dout=dout, dsT=dsT)


def test_gradient_in_place_and_optional_outputs():
    """The C entry point: ds0 may be dsT, or absent."""
    import ctypes
    T = 1500
    x, dout, dsT = make(T, 1, 1, 2, 64, 64, "fp16")
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    st = L.gdr_forward(**x, save=True)
    want = L.gdr_backward(st, *five, dout=dout, dsT=dsT)
    opt = L.GdrOptions(None, 64 ** -0.5)
    ws = L.empty_workspace(L.gdr_bwd_workspace_size(st.dims), "cuda")
    for ds in ("in place", None):
        g, d = L.GdrGrads(st.dims, torch.float16, "cuda"), dsT.clone()
        p = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        rc = L.load().lstm_gdr_bwd(ctypes.byref(st.dims), ctypes.byref(opt), p(dout), p(d), p(x["q"]), p(x["k"]), None, p(x["g"]),
                                   p(x["beta"]), p(st.states), p(st.deltas), p(g.dq), p(g.dk), p(g.dv), p(g.dg), p(g.dbeta),
                                   p(d) if ds else None, None, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == L.LSTM_OK
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(getattr(g, n), getattr(want, n))
        assert torch.equal(d, want.ds0 if ds else dsT)
    assert L.lstm_status(ws) == L.LSTM_OK


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,V", [(64, 64, 72), (128, 128, 136), (50, 64, 8)])
def test_outputs_where_large_parts_cancel(T, K, V, dt):
    """A large state overwritten token by token: o_t = v_t is the sum of q S0 and P U, each thousands of times as large.

    Keys and queries are unit vectors, so that every product has one term: besides the rounding to the output's type
    only v - S0, the sum and what an accumulator's alignment drops are rounded, 8 steps of 2^-24 of the parts at most."""
    gen = torch.Generator(device="cuda").manual_seed(T + V)
    k = torch.eye(K, device="cuda")[:T].to(DT[dt]).view(T, 1, 1, K)
    v = torch.randn(T, 1, 1, V, generator=gen, device="cuda").to(DT[dt])
    s0 = 1e4 * torch.randn(1, 1, K, V, generator=gen, device="cuda")
    st = L.gdr_forward(k, k, v, torch.zeros(T, 1, 1, device="cuda"), torch.ones(T, 1, 1, device="cuda"), s0, scale=1.0, save=True)
    err = (st.o.double() - v.double()).abs()[:, 0, 0]
    parts = s0[0, 0, :T].double().abs() + v.double().abs()[:, 0, 0]
    assert bool((err <= torch.finfo(DT[dt]).eps / 2 * v.double().abs()[:, 0, 0] + 8 * 2.0 ** -24 * parts).all()), float((err / parts).max())


def test_options_of_another_forward():
    """A backward whose scale or lengths are not its forward's would mix two problems (P and the gates are the forward's)."""
    x, dout, dsT = make(100, 3, 1, 2, 64, 64, "bf16")
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    lengths = torch.tensor([100, 7, 64], dtype=torch.int32, device="cuda")
    kw = dict(dout=dout, dsT=dsT)
    for st in (L.gdr_forward(**x, save=True, scale=0.5, lengths=lengths),
               L.gdr_forward(**x, save=True, scale=0.5, lengths=lengths, ws=L.empty_workspace(L.gdr_fwd_workspace_size(L.gdr_dims(100, 3, 1, 2, 64, 64, torch.bfloat16), True), "cuda"))):
        want = L.gdr_backward(st, *five, **kw, scale=0.5, lengths=lengths)
        for scale in (None, 0.25, 0.5001):
            with pytest.raises(ValueError, match="scale"):
                L.gdr_backward(st, *five, **kw, scale=scale, lengths=lengths)
        for other in (None, lengths.flip(0), lengths + 1):
            with pytest.raises(ValueError, match="lengths"):
                L.gdr_backward(st, *five, **kw, scale=0.5, lengths=other)
        copy = L.gdr_backward(st, *five, **kw, scale=0.5, lengths=lengths.clone())  # the same lengths in another tensor
        assert torch.equal(copy.dk, want.dk) and torch.equal(copy.dg, want.dg)
    st = L.gdr_forward(**x, save=True)
    assert torch.equal(L.gdr_backward(st, *five, **kw, scale=64 ** -0.5).dq, L.gdr_backward(st, *five, **kw).dq)
    with pytest.raises(ValueError, match="lengths"):
        L.gdr_backward(st, *five, **kw, lengths=lengths)
    graph = torch.cuda.CUDAGraph()
    copy = lengths.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st = L.gdr_forward(**x, save=True, lengths=lengths)
        gr = L.gdr_backward(st, *five, **kw, lengths=lengths)
        with pytest.raises(ValueError, match="own lengths"):
            L.gdr_backward(st, *five, **kw, lengths=copy)
    graph.replay()
    torch.cuda.synchronize()
    st = L.gdr_forward(**x, save=True, lengths=lengths)
    assert torch.equal(gr.dk, L.gdr_backward(st, *five, **kw, lengths=lengths).dk)


def off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


@pytest.mark.parametrize("shape", [(256, 2, 1, 2, 128, 128), (512, 1, 2, 2, 64, 64), (600, 1, 1, 1, 96, 72)], ids=str)
def test_state_gradient_as_close_as_a_float_sum(shape):
    """ds0 in norm.  A tensor core's accumulator drops what lies below its last place, half a unit (2^-24) on average, at
    every step that meets the full sum: the 8 steps of the two large products, if every small one comes before them."""
    x, dout, dsT = make(*shape, "fp32")
    d = {n: t.double().requires_grad_() for n, t in x.items()}
    o, S = reference(**d, lengths=None, scale=shape[4] ** -0.5)
    want, = torch.autograd.grad((o * dout.double()).sum() + (S * dsT.double()).sum(), [d["s0"]])
    st = L.gdr_forward(**x, save=True)
    gr = L.gdr_backward(st, *(x[n] for n in ("q", "k", "v", "g", "beta")), dout=dout, dsT=dsT)
    assert off(gr.ds0, want) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("shape,dt", [((2050, 1, 1, 1, 128, 128), "fp32"), ((1500, 2, 1, 2, 64, 40), "fp32"), ((900, 1, 1, 2, 96, 256), "fp32"),
                                      ((3000, 1, 2, 2, 128, 136), "bf16"), ((1100, 3, 1, 1, 128, 72), "fp16")], ids=str)
def test_segments_against_pieces(shape, dt):
    """What passes from segment to segment where little is forgotten: a split call is the same sequence in pieces of three
    chunks (too short to split), the state and its gradient handed on.

    In norm.  A chunk's or a joint's sums lose 8 half units of a float (see above), the same share of the state in both
    forms but for their order; over the 12 chunks of a segment at most 96 * 2^-24 < 2^-17.  A transition matrix short of
    its second terms would be off by 2^-9."""
    T = shape[0]
    d, piece = (L.gdr_dims(t, *shape[1:], DT[dt]) for t in (T, 192))
    assert L.gdr_fwd_workspace_size(d) - 256 > -(-T // 64) / 3 * (L.gdr_fwd_workspace_size(piece) - 256)  # it is split
    x, dout, dsT = make(*shape, dt)
    x["g"] *= 0.002
    x["beta"] *= 0.1
    names = ("q", "k", "v", "g", "beta")
    one = L.gdr_forward(**x, save=True)
    gone = L.gdr_backward(one, *(x[n] for n in names), dout=dout, dsT=dsT)
    s0, parts = x["s0"], []
    for t in range(0, T, 192):
        y = [x[n][t:t + 192] for n in names]
        parts.append((L.gdr_forward(*y, s0=s0, save=True), y, dout[t:t + 192]))
        s0 = parts[-1][0].sT
    ds, grads = dsT, []
    for st, y, do in reversed(parts):
        grads.insert(0, L.gdr_backward(st, *y, dout=do, dsT=ds))
        ds = grads[0].ds0
    assert off(one.sT, s0) <= 2.0 ** -17 and off(gone.ds0, ds) <= 2.0 ** -17
    assert off(one.states[len(one.states) - 1], parts[-1][0].states[-1]) <= 2.0 ** -17
    half = torch.finfo(DT[dt]).eps / 2 if dt != "fp32" else 0  # (two roundings to the type may differ by a step)
    assert off(one.o, torch.cat([st.o for st, _, _ in parts])) <= 2.0 ** -17 + half
    for n in ("dq", "dk", "dv"):
        assert off(getattr(gone, n), torch.cat([getattr(g, n) for g in grads])) <= 2.0 ** -16 + half
    for n in ("dg", "dbeta"):
        assert off(getattr(gone, n), torch.cat([getattr(g, n) for g in grads])) <= 2.0 ** -16


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [9, 100, 1500])
def test_state_of_a_sequence_without_tokens(T, dt):
    """NaN and infinities in the state (or its gradient) of an empty place of the batch stay there, bit by bit; its outputs
    and gradients are zero and the other sequences' what they were."""
    x, dout, dsT = make(T, 3, 1, 2, 64, 72, dt)
    lengths = torch.tensor([T, 0, T - 1], dtype=torch.int32, device="cuda")
    names = ("q", "k", "v", "g", "beta")

    def run(x, dsT):
        few = L.gdr_forward(**x, lengths=lengths)
        st = L.gdr_forward(**x, lengths=lengths, save=True)
        return few, st, L.gdr_backward(st, *(x[n] for n in names), dout=dout, dsT=dsT, lengths=lengths)

    want = run(x, dsT)
    y, ds = {n: t.clone() for n, t in x.items()}, dsT.clone()
    y["s0"][1, 0, 3, ::5] = float("nan")
    y["s0"][1, 1, ::7] = float("inf")
    ds[1, 0, ::9] = float("nan")
    got = run(y, ds)
    bits = lambda t: t.view(torch.int32)  # noqa: E731
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a.o, b.o) and torch.equal(a.sT[::2], b.sT[::2]) and torch.equal(bits(a.sT[1]), bits(y["s0"][1]))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        g = getattr(got[2], n)
        assert torch.equal(g, getattr(want[2], n)) and not g[:, 1].any(), n
    assert torch.equal(got[2].ds0[::2], want[2].ds0[::2]) and torch.equal(bits(got[2].ds0[1]), bits(ds[1]))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [9, 100, 1500])
def test_state_of_a_sequence_without_tokens(T, dt):
    """NaN and infinities in the state (or its gradient) of an empty place of the batch stay there, bit by bit; its outputs
    and gradients are zero and the other sequences' what they were."""
    x, dout, dsT = make(T, 3, 1, 2, 64, 72, dt)
    lengths = torch.tensor([T, 0, T - 1], dtype=torch.int32, device="cuda")
    names = ("q", "k", "v", "g", "beta")

    def run(x, dsT):
        few = L.gdr_forward(**x, lengths=lengths)
        st = L.gdr_forward(**x, lengths=lengths, save=True)
        return few, st, L.gdr_backward(st, *(x[n] for n in names), dout=dout, dsT=dsT, lengths=lengths)

    want = run(x, dsT)
    y, ds = {n: t.clone() for n, t in x.items()}, dsT.clone()
    y["s0"][1, 0, 3, ::5] = float("nan")
    y["s0"][1, 1, ::7] = float("inf")
    ds[1, 0, ::9] = float("nan")
    got = run(y, ds)
    bits = lambda t: t.view(torch.int32)  # noqa: E731
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a.o, b.o) and torch.equal(a.sT[::2], b.sT[::2]) and torch.equal(bits(a.sT[1]), bits(y["s0"][1]))
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        g = getattr(got[2], n)
        assert torch.equal(g, getattr(want[2], n)) and not g[:, 1].any(), n
    assert torch.equal(got[2].ds0[::2], want[2].ds0[::2]) and torch.equal(bits(got[2].ds0[1]), bits(ds[1]))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(300, 4, 1, 3, 40, 136), (1500, 3, 1, 1, 64, 64), (260, 40, 2, 4, 128, 24)], ids=str)
def test_chunks_of_padding(shape, dt):
    """Sequences that end chunks before the longest (in other segments of a split one): as the same sequences alone, padding
    zero, the kept states those of the end."""
    x, dout, dsT = make(*shape, dt)
    T, B = shape[:2]
    lengths = torch.tensor([(T, 1, 64, 65, 130, T - 64, 0)[b % 7] for b in range(B)], dtype=torch.int32, device="cuda")
    st, gr = check(x, dout, dsT, lengths=lengths)
    for b, n in enumerate(lengths.tolist()):
        for t in (st.o, gr.dq, gr.dk, gr.dv, gr.dg, gr.dbeta):
            assert not t[n:, b].any()
        for c in range(-(-n // 64), -(-T // 64)):
            assert torch.equal(st.states[c, b], st.sT[b])


def test_lengths_change_between_replays():
    """A captured step reads its lengths when it is replayed: whole chunks of padding come and go."""
    x, dout, dsT = make(1500, 3, 1, 2, 64, 72, "bf16")
    names = ("q", "k", "v", "g", "beta")
    five = [x[n] for n in names]
    lengths = torch.tensor([1500, 1500, 1500], dtype=torch.int32, device="cuda")
    L.gdr_forward(**x, save=True, lengths=lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = L.gdr_forward(**x, save=True, lengths=lengths)
        gr = L.gdr_backward(st, *five, dout=dout, dsT=dsT, lengths=lengths)
    for now in ([1500, 0, 64], [65, 1400, 1], [0, 0, 0], [1500, 1500, 1500]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = L.gdr_forward(**x, save=True, lengths=lengths)
        wg = L.gdr_backward(want, *five, dout=dout, dsT=dsT, lengths=lengths)
        assert torch.equal(st.o, want.o) and torch.equal(st.sT, want.sT) and torch.equal(st.states, want.states)
        for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
            assert torch.equal(getattr(gr, n), getattr(wg, n)), (now, n)
