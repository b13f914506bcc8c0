"""lstm_logprob_fwd / lstm_logprob_bwd against plain formulas in 64 bits.

Tolerances.  An exponential has a relative error of about 2^-22 (the
instruction) + |x - m| 2^-23 (its argument, below 100 here: 2^-16.3 where it
matters least, since e^-100 is nothing; terms that carry weight have
|x - m| below 20), so sums are within 2^-18, and their logarithms within 2^-18
absolutely; log p and the entropy add roundings of 2^-24 of terms below 100."""
import math

import pytest
import torch

from backward_lstm_fwd_b200 import binding as L
from backward_lstm_fwd_b200 import build as lbuild

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ABS = 2.0 ** -18 + 100 * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    lbuild.build()


def reference(logits, targets, temperature):
    z = logits.double() / temperature
    z = z - z.amax(1, keepdim=True)  # first: beside the lowest float a log-sum would vanish even in 64 bits
    lp = z - torch.log(torch.exp(z).sum(1, keepdim=True))
    p = torch.exp(lp)
    h = -torch.where(p > 0, p * lp, torch.zeros((), dtype=torch.float64, device=z.device)).sum(1)
    t = targets.long()
    ok = (t >= 0) & (t < logits.shape[1])
    tl = torch.where(ok, lp.gather(1, t.clamp(0, logits.shape[1] - 1)[:, None])[:, 0], torch.zeros((), dtype=torch.float64, device=z.device))
    return lp, p, h, tl, ok


def reference_grad(lp, p, h, t, ok, dlogp, dh, temperature):
    hot = torch.zeros_like(p)
    hot[torch.arange(len(t), device=t.device)[ok], t.long()[ok]] = 1.0
    dl = torch.where(ok, dlogp.double(), torch.zeros((), dtype=torch.float64, device=p.device))[:, None]
    inner = torch.where(p > 0, p * (lp + h[:, None]), torch.zeros((), dtype=torch.float64, device=p.device))
    return (dl * (hot - p) - dh.double()[:, None] * inner) / temperature


def check(logits, targets, top, temperature, grads=True):
    N, V = logits.shape
    st = L.logprobs(logits, targets, top=top, temperature=temperature)
    lp, p, h, tl, ok = reference(logits, targets, temperature)
    fin = torch.isfinite(tl)
    assert torch.equal(torch.isfinite(st.logp), fin)
    assert bool(((st.logp.double() - tl).abs()[fin] <= ABS).all())
    assert bool(((st.entropy.double() - h).abs() <= ABS * (1 + h)).all())
    assert bool(((st.lse.double() - torch.logsumexp(logits.double() / temperature, 1)).abs() <= ABS + 2.0 ** -22 * logits.double().abs().amax(1) / temperature).all())
    if top:
        order = torch.argsort(-logits.double(), dim=1, stable=True)[:, :top]
        assert torch.equal(st.top_ids.long(), order)
        want = lp.gather(1, order)
        f = torch.isfinite(want)
        assert torch.equal(torch.isfinite(st.top_logp), f)
        assert bool(((st.top_logp.double() - want).abs()[f] <= ABS).all())
    if grads:
        dlogp, dh = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
        d = L.logprobs_backward(st, logits, targets, dlogp=dlogp, dentropy=dh, temperature=temperature)
        want = reference_grad(lp, p, h, targets, ok, dlogp, dh, temperature)
        assert d.stride() == logits.stride() or N == 1
        # p is within 2^-18 of itself, the factor (log p + entropy) within ABS (1 + h); one rounding to the type
        mag = (dlogp.double().abs()[:, None] * (p + (want != 0)) + dh.double().abs()[:, None] * p * (torch.where(p > 0, lp, torch.zeros_like(lp)).abs() + h[:, None] + 1)) / temperature
        tol = (2 * ABS) * mag + torch.finfo(d.dtype).eps / 2 * want.abs() + 2.0 ** -24
        assert bool(((d.double() - want).abs() <= tol).all())
    return st


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,V,pad,top", [(1, 1, 0, 1), (3, 2, 1, 2), (2, 7, 0, 7), (5, 63, 2, 20), (4, 4095, 1, 5),
                                         (1, 128000, 0, 20), (3, 50001, 7, 64), (700, 1003, 5, 8), (2, 9000, 0, 0),
                                         (301, 5000, 3, 1), (20, 40000, 3, 5), (37, 70001, 1, 17), (37, 70001, 1, 0),
                                         (150, 30000, 5, 16), (18, 33000, 0, 64), (19, 33000, 0, 33)])
def test_against_64_bits(N, V, pad, top, dt):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    logits = (4 * torch.randn(N, V + pad, generator=g, device="cuda")).to(DT[dt])[:, :V]
    targets = torch.randint(0, V, (N,), generator=g, device="cuda")
    check(logits, targets, top, 0.8)
    check(logits, targets.int(), top, 1.0, grads=False)


def test_ignored_targets():
    logits = torch.randn(4, 300, device="cuda")
    targets = torch.tensor([-1, 300, 5, -100], device="cuda")
    st = check(logits, targets, 2, 1.0)
    assert st.logp[[0, 1, 3]].abs().sum() == 0
    d = L.logprobs_backward(st, logits, targets, dlogp=torch.ones(4, device="cuda"))
    assert not d[[0, 1, 3]].any() and d[2].any()


@pytest.mark.parametrize("dt", list(DT))
def test_masks(dt):
    """-inf and lowest-value masks, rows with one or no choice left."""
    N, V = 8, 3001
    x = torch.randn(N, V, device="cuda").to(DT[dt])
    inf = float("-inf")
    x[0, ::2] = inf
    x[1, :] = inf
    x[2, :] = inf
    x[2, 17] = 1.5
    x[3, :2000] = inf  # whole batches of masked elements first
    x[4, 5:] = torch.finfo(DT[dt]).min
    x[5, :] = torch.finfo(DT[dt]).min
    x[6, :-1] = torch.finfo(DT[dt]).min
    t = torch.tensor([0, 3, 17, 2500, 2, 9, V - 1, 1], device="cuda")
    st = L.logprobs(x, t, top=4, temperature=1.0)
    rows = [0, 2, 3, 4, 5, 6, 7]
    lp, p, h, tl, ok = reference(x[rows], t[rows], 1.0)
    f = torch.isfinite(tl)
    assert torch.equal(torch.isfinite(st.logp[rows]), f)
    assert bool(((st.logp[rows].double() - tl).abs()[f] <= ABS).all())
    assert bool(((st.entropy[rows].double() - h).abs() <= ABS * (1 + h)).all())
    assert st.logp[1] == inf and st.entropy[1] == 0 and bool((st.top_logp[1] == inf).all())
    assert st.top_ids[1].tolist() == [0, 1, 2, 3] and st.top_ids[2].tolist() == [17, 0, 1, 2] and st.top_ids[5].tolist() == [0, 1, 2, 3]
    d = L.logprobs_backward(st, x, t, dlogp=torch.ones(N, device="cuda"), dentropy=torch.ones(N, device="cuda"))
    assert bool(torch.isfinite(d).all()) and not d[1].any()
    want = reference_grad(lp, p, h, t[rows], ok, torch.ones(7, device="cuda"), torch.ones(7, device="cuda"), 1.0)
    assert bool(((d[rows].double() - want).abs() <= 4 * ABS * (1 + h[:, None]) + torch.finfo(DT[dt]).eps / 2 * want.abs()).all())


def test_nan_and_infinity():
    x = torch.randn(4, 600, device="cuda")
    x[0, 7] = float("nan")
    x[1, 9] = float("inf")
    x[2, 590:] = float("nan")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    st = L.logprobs(x, t, top=3)
    assert bool(torch.isnan(st.logp[:3]).all()) and bool(torch.isnan(st.entropy[:3]).all())
    assert bool(torch.isfinite(st.logp[3]))
    assert st.top_ids[1, 0] == 9 and 7 not in st.top_ids[0].tolist()
    d = L.logprobs_backward(st, x, t, dlogp=torch.ones(4, device="cuda"))
    assert bool(torch.isnan(d[0]).any()) and bool(torch.isfinite(d[3]).all())


@pytest.mark.parametrize("N", [2, 400])
def test_equal_values(N):
    """Rows of equal values: more candidates than the list holds; the lowest indices win."""
    for x in (torch.zeros(N, 20000, device="cuda"), torch.full((N, 20000), -3.0, device="cuda").bfloat16()):
        x[:, 11111] = 1.0
        st = L.logprobs(x, top=5)
        assert st.top_ids[N - 1].tolist() == [11111, 0, 1, 2, 3]
        assert st.logp is None
    y = torch.zeros(N, 20000, device="cuda")
    y[:, ::2] = -0.0  # the zeros are equal
    assert L.logprobs(y, top=3).top_ids[0].tolist() == [0, 1, 2]


@pytest.mark.parametrize("N", [2, 20, 400])
@pytest.mark.parametrize("step", [1, -1])
def test_sorted_rows(N, step):
    """Rows that rise make every element a candidate (the list overflows), rows that fall the first ones alone."""
    x = (torch.arange(40000, device="cuda", dtype=torch.float32) * (step * 1e-3)).repeat(N, 1)
    for top in (1, 16, 20):
        st = L.logprobs(x, top=top)
        want = torch.arange(top, device="cuda") if step < 0 else 39999 - torch.arange(top, device="cuda")
        assert bool((st.top_ids == want).all())
        check(x, torch.arange(N, device="cuda"), top, 1.0)


def test_confident_row():
    """A row whose target has all but 2e-6 of the weight: log p and the entropy to the last digits of a 32-bit sum near one.

    The maximum's 1 enters one thread's sum; every later addition to it rounds by 2^-24 at most: 3 more of the thread's
    own 4 elements, 5 shuffles, 7 warps, and the logarithm's result: 16 roundings."""
    x = torch.zeros(1, 1000, device="cuda")
    x[0, 3] = 20.0
    st = L.logprobs(x, torch.tensor([3], device="cuda"))
    rest = 999 * math.exp(-20.0)
    assert abs(float(st.logp) + math.log1p(rest)) <= 16 * 2.0 ** -24
    assert abs(float(st.entropy) - (math.log1p(rest) + 20 * rest / (1 + rest))) <= 16 * 2.0 ** -24 + 2.0 ** -18 * 20 * rest


def test_in_place_and_out():
    x = torch.randn(40, 777, device="cuda").half()
    t = torch.randint(0, 777, (40,), device="cuda")
    dl = torch.randn(40, device="cuda")
    st = L.logprobs(x, t, temperature=2.0)
    want = L.logprobs_backward(st, x, t, dlogp=dl, temperature=2.0)
    odd = torch.full((40, 780), 9.0, device="cuda", dtype=torch.half)
    got = L.logprobs_backward(st, x, t, dlogp=dl, temperature=2.0, out=odd[:, :777])
    assert torch.equal(got, want) and bool((odd[:, 777:] == 9).all())
    L.logprobs_backward(st, x, t, dlogp=dl, temperature=2.0, out=x)
    assert torch.equal(x, want)


def test_gradient_by_differences():
    """The gradient of <a, logp> + <b, entropy> against central differences in 64 bits."""
    N, V, temperature, eps = 3, 9, 0.7, 1e-5
    x = torch.randn(N, V, device="cuda")
    t = torch.tensor([2, 0, 8], device="cuda")
    a, b = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    st = L.logprobs(x, t, temperature=temperature)
    d = L.logprobs_backward(st, x, t, dlogp=a, dentropy=b, temperature=temperature).double()

    def loss(y):
        z = y / temperature
        lp = torch.log_softmax(z, 1)
        return (a.double() * lp[torch.arange(N), t]).sum() - (b.double()[:, None] * lp.exp() * lp).sum()

    for r in range(N):
        for c in range(V):
            e = torch.zeros(N, V, dtype=torch.float64, device="cuda")
            e[r, c] = eps
            # truncation about eps^2, cancellation about 2^-52 / eps
            assert abs(float((loss(x.double() + e) - loss(x.double() - e)) / (2 * eps)) - float(d[r, c])) <= 1e-5


def test_empty_streams_and_graphs():
    assert L.logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=2).logp.shape == (0,)
    N, V = 3, 40000
    x, t = torch.randn(N, V, device="cuda"), torch.randint(0, V, (N,), device="cuda")
    want = L.logprobs(x, t, top=6)
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs.append(L.logprobs(x, t, top=6))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.logp, want.logp) and torch.equal(o.top_ids, want.top_ids) and torch.equal(o.entropy, want.entropy)
    xb, tb = torch.zeros_like(x), torch.zeros_like(t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = L.logprobs(xb, tb, top=6)
        d = L.logprobs_backward(st, xb, tb, dlogp=st.entropy)
    xb.copy_(x)
    tb.copy_(t)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(st.logp, want.logp) and torch.equal(st.top_ids, want.top_ids)
    assert torch.equal(d, L.logprobs_backward(want, x, t, dlogp=want.entropy))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N", [3, 400])
def test_masked_parts(N, dt):
    """Long rows that blocks share, whole parts of them masked, -inf and the lowest value side by side."""
    V = 70000
    low, inf = torch.finfo(DT[dt]).min, float("-inf")
    x = torch.randn(N, V, device="cuda").to(DT[dt])
    x[0, :60000] = inf
    x[1, 5000:] = low
    x[2] = inf
    x[2, 100:20000:7] = low
    t = torch.tensor([65000, 17, 107], device="cuda").repeat(N // 3 + 1)[:N]
    st = L.logprobs(x, t, top=3)
    n = (20000 - 100 + 6) // 7
    assert abs(float(st.logp[2]) + math.log(n)) <= ABS and abs(float(st.entropy[2]) - math.log(n)) <= ABS * 10
    assert st.top_ids[2].tolist() == [100, 107, 114]
    keep = [0, 1] + list(range(3, N))
    _, _, h, tl, _ = reference(x[keep], t[keep], 1.0)
    assert bool(((st.logp[keep].double() - tl).abs() <= ABS).all())
    assert bool(((st.entropy[keep].double() - h).abs() <= ABS * (1 + h)).all())
    d = L.logprobs_backward(st, x, t, dlogp=torch.ones(N, device="cuda"))
    assert bool(torch.isfinite(d).all()) and not d[0, :60000].any() and not d[2, 1:100].any()
    assert abs(float(d[2, 114]) + 1 / n) <= 2 * ABS / n + torch.finfo(d.dtype).eps / 2 / n + 2.0 ** -24


@pytest.mark.parametrize("dt", list(DT))
def test_rows_from_anywhere(dt):
    """Slices of rows, targets and gradients that start at no 16-byte boundary."""
    x = torch.randn(9, 1001, device="cuda").to(DT[dt])
    t = torch.randint(0, 1001, (9,), device="cuda", dtype=torch.int32)
    dl = torch.randn(9, device="cuda")
    want = L.logprobs(x, t, top=4)
    dw = L.logprobs_backward(want, x, t, dlogp=dl)
    for r in range(1, 9):
        st = L.logprobs(x[r:], t[r:], top=4)
        assert bool(((st.logp - want.logp[r:]).abs() <= ABS).all()) and torch.equal(st.top_ids, want.top_ids[r:])
        d = L.logprobs_backward(st, x[r:], t[r:], dlogp=dl[r:])
        assert bool(((d.double() - dw[r:].double()).abs() <= 4 * ABS + torch.finfo(d.dtype).eps * dw[r:].double().abs()).all())
    cols = x[:, 3:900]
    st = L.logprobs(cols, top=2)
    assert torch.equal(st.top_ids, L.logprobs(cols.contiguous(), top=2).top_ids)


def check_large(x, t, top, temperature):
    """check() where log p may be large: it takes four roundings of its size more (x - m, 1 / temperature, their product,
    the sum), the logarithm of the sum one of the largest z; beyond a float's range it is infinite."""
    N = len(x)
    st = L.logprobs(x, t, top=top, temperature=temperature)
    lp, p, h, tl, ok = reference(x, t, temperature)

    def near(got, want):
        fits = torch.isfinite(want.float())
        assert torch.equal(torch.isfinite(got), fits) and bool((got[~fits] == want.float()[~fits]).all())
        assert bool(((got.double() - want).abs()[fits] <= ABS + 2.0 ** -22 * want.abs()[fits]).all())

    near(st.logp, tl)
    assert bool(((st.entropy.double() - h).abs() <= ABS * (1 + h)).all())
    z = x.double() / temperature
    big = z.abs().amax(1) > 1e38
    assert bool(((st.lse.double() - torch.logsumexp(z, 1)).abs()[~big] <= ABS + 2.0 ** -22 * z.abs().amax(1)[~big]).all())
    if top:
        order = torch.argsort(-x.double(), dim=1, stable=True)[:, :top]
        assert torch.equal(st.top_ids.long(), order)
        near(st.top_logp, lp.gather(1, order))
    dlogp, dh = (temperature * torch.randn(N, device="cuda") for _ in range(2))
    d = L.logprobs_backward(st, x, t, dlogp=dlogp, dentropy=dh, temperature=temperature)
    want = reference_grad(lp, p, h, t, ok, dlogp, dh, temperature)
    mag = (dlogp.double().abs()[:, None] * (p + (want != 0)) + dh.double().abs()[:, None] * p * (lp.abs().clamp(max=1e30) + h[:, None] + 1)) / temperature
    assert bool(((d.double() - want).abs() <= 2 * ABS * mag + torch.finfo(d.dtype).eps / 2 * want.abs() + 2.0 ** -24).all())


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("temperature", [1.0, 0.3, 0.1])
@pytest.mark.parametrize("value", [-1e5, -3e7, -1e9, -1e10, -1e12, -1e15, -3e38])
def test_masks_of_any_value(value, temperature, dt):
    """Finite masks from small ones to the lowest: a range, scattered, all but one, all; rows in one block and shared."""
    for N, V, top in ((6, 3001, 3), (6, 3001, 0), (6, 70001, 4), (6, 70001, 20), (300, 3001, 0), (300, 3001, 5)):
        g = torch.Generator(device="cuda").manual_seed(N + V + top)
        x = (3 * torch.randn(N, V, generator=g, device="cuda")).to(DT[dt])
        x[0, : V * 3 // 4] = value
        x[1, ::2] = value
        x[2, :] = value
        x[2, V // 3] = 2.5
        x[3, :] = value
        x[4, 100:] = value
        check_large(x, torch.tensor([V - 3, 0, V // 3, 5, 200, 7], device="cuda").repeat(N // 6 + 1)[:N], top, temperature)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt,size,temperature", [("fp32", 1e7, 1.0), ("fp32", 2e9, 1.0), ("fp32", 3e12, 1.0), ("fp32", 1e17, 0.5),
                                                 ("bf16", 1e10, 1.0), ("bf16", 3e38, 1.0), ("fp16", 3000.0, 1e-5),
                                                 ("fp16", 60000.0, 1e-6), ("fp32", 700.0, 1e-6), ("fp32", 1e30, 1e-6),
                                                 ("fp32", 1e12, 1e6), ("fp32", 3e38, 1e6)])
def test_large_logits(dt, size, temperature, sign):
    """Rows of large logits, a few steps of their type or a factor of two apart, or all equal."""
    for N, V, top in ((4, 2050, 3), (4, 70001, 0), (4, 70001, 17), (300, 2050, 0)):
        g = torch.Generator(device="cuda").manual_seed(V + top)
        steps = 1 + torch.randint(0, 4, (N, V), generator=g, device="cuda") * torch.finfo(DT[dt]).eps
        spread = 0.5 + 0.5 * torch.rand(N, V, generator=g, device="cuda")
        x = (sign * size * 0.9 * torch.where(torch.arange(N, device="cuda")[:, None] % 2 == 0, steps, spread)).to(DT[dt])
        x[3] = x[3, 0]
        check_large(x, torch.randint(0, V, (N,), generator=g, device="cuda"), top, temperature)


@pytest.mark.parametrize("dt", list(DT))
def test_masked_logits_under_a_large_entropy_gradient(dt):
    """p = 0 has no gradient, however large that of the entropy (a scaled loss, a low temperature)."""
    x = torch.randn(3, 700, device="cuda").to(DT[dt])
    x[:, 5:300] = float("-inf")
    x[1, 400:] = torch.finfo(DT[dt]).min
    dh = torch.tensor([65536.0, 1e12, -3e14], device="cuda")
    for temperature in (1.0, 1e-6):
        st = L.logprobs(x, temperature=temperature)
        d = L.logprobs_backward(st, x, dentropy=dh, temperature=temperature)
        assert not d[:, 5:300].any() and not torch.isnan(d).any()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("V", [1000, 1001])
def test_gradient_of_rows_far_apart(V, dt):
    """The last step's logits of a [B, T, V] tensor, one sequence of a [T, B, V] one: the gradient holds no more than itself."""
    wide = torch.randn(6, 50, V, device="cuda").to(DT[dt])
    t = torch.randint(0, V, (6,), device="cuda")
    dl = torch.randn(6, device="cuda")
    for x in (wide[:, -1], wide[:, 0], wide[1:6, 7]):
        n = len(x)
        st = L.logprobs(x, t[:n])
        d = L.logprobs_backward(st, x, t[:n], dlogp=dl[:n])
        assert d.untyped_storage().nbytes() <= n * (V + 8) * d.element_size()
        out = torch.empty_like(d).contiguous()
        L.logprobs_backward(st, x, t[:n], dlogp=dl[:n], out=out)
        assert torch.equal(d, out)
    padded = wide.view(6, -1)[:, : V - 60]  # (of rows far apart too)
    assert L.logprobs_backward(L.logprobs(padded), padded).stride(0) < V
    near = wide.view(300, V)[:, : V - 60]  # a padded vocabulary keeps its stride
    assert L.logprobs_backward(L.logprobs(near), near).stride() == near.stride()


@pytest.mark.parametrize("top", [-1, -5, 65, 1 << 40])
def test_number_of_alternatives_is_refused_first(top):
    """Before outputs of that many are allocated (or their number is cut to an int)."""
    with pytest.raises(L.LstmError, match="lstm_logprob_fwd"):
        L.logprobs(torch.randn(2, 100, device="cuda"), top=top)


def test_state_of_another_forward():
    """Rows of another width (a padded vocabulary, or the same without its padding) are another softmax."""
    x = torch.randn(5, 120, device="cuda")
    st = L.logprobs(x[:, :100])
    for y in (x, x[:, :99], x[:4, :100]):
        with pytest.raises(ValueError):
            L.logprobs_backward(st, y, dentropy=torch.ones(len(y), device="cuda"))
    with pytest.raises(ValueError, match="temperature"):
        L.logprobs_backward(st, x[:, :100], dentropy=torch.ones(5, device="cuda"), temperature=2.0)
