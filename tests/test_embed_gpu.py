"""lstm_embed_fwd / lstm_embed_bwd against plain formulas in 64 bits.

Tolerances: x is one product rounded to float and once more to the type; the
gradient is a float sum of n terms and a product (n + 1 roundings of 2^-24 of
the sum of magnitudes, at most)."""
import pytest
import torch

from backward_lstm_fwd_b200 import binding as L
from backward_lstm_fwd_b200 import build as lbuild

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    lbuild.build()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def make_ids(n, vocab, seed, kind, dtype):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        ids = torch.randint(-2, vocab + 2, (n,), generator=g)
    elif kind == "same":
        ids = torch.full((n,), vocab - 1)
    elif kind == "padding":
        ids = torch.full((n,), -1)
    else:  # a few heavy tokens among rare ones
        ids = torch.exp(torch.rand(n, generator=g) * torch.log(torch.tensor(float(vocab)))).long() - 1
        ids[torch.rand(n, generator=g) < 0.1] = vocab // 2
    return ids.to(dtype).cuda()


def expect(ids, dx, vocab, scale):
    """(sum, sum of magnitudes) of the table's gradient in float64."""
    i = ids.long().reshape(-1)
    ok = (i >= 0) & (i < vocab)
    d = dx.double().reshape(len(i), dx.shape[-1])[ok]
    out = torch.zeros(vocab, dx.shape[-1], dtype=torch.float64, device=dx.device)
    mag = out.clone().index_add_(0, i[ok], d.abs())
    return out.index_add_(0, i[ok], d) * scale, mag * abs(scale)


def check_grad(got, ids, dx, vocab, scale):
    ref, mag = expect(ids, dx, vocab, scale)
    n = int(torch.bincount(ids.long().reshape(-1).clamp(0, vocab), minlength=1).max()) if ids.numel() else 0
    # pairwise at best, one after another at worst: n + 2 roundings
    assert bool(((got.double() - ref).abs() <= (n + 2) * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,vocab,I", [(1, 1, 1), (1, 7, 8), (33, 50, 24), (128, 1000, 1024), (5, 9, 7),
                                       (4097, 513, 260), (700, 33, 2050)])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_lookup(n, vocab, I, dt, idt):
    ids = make_ids(n, vocab, n, "uniform", idt)
    table = torch.randn(vocab, I, device="cuda").to(DT[dt])
    scale = 1.7
    x = L.embed(ids, table, scale)
    ok = (ids >= 0) & (ids < vocab)
    ref = torch.where(ok[:, None], table.double()[ids.long().clamp(0, vocab - 1)] * float(torch.tensor(scale)), 0.0)
    tol = 2.0 ** -24 + half_step(DT[dt]) + 2.0 ** -22
    assert bool(((x.double() - ref).abs() <= tol * ref.abs() + 2.0 ** -25).all())
    same = L.embed(ids, table, 1.0)  # a scale of one keeps every bit
    assert torch.equal(same, torch.where(ok[:, None], table[ids.long().clamp(0, vocab - 1)], torch.zeros((), dtype=DT[dt], device="cuda")))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["uniform", "same", "heavy", "padding"])
@pytest.mark.parametrize("n,vocab,I", [(1, 1, 4), (1, 40, 3), (31, 9, 8), (32, 9, 8), (33, 700, 260), (64, 2, 12),
                                       (2048, 513, 16), (2049, 600, 20), (5000, 262150, 8), (9000, 77, 1028)])
def test_gradient(n, vocab, I, kind, dt):
    ids = make_ids(n, vocab, n + 1, kind, torch.int64)
    dx = torch.randn(n, I, device="cuda").to(DT[dt])
    got = L.embed_backward(ids, dx, vocab, scale=0.5, out=torch.full((vocab, I), 7.0, device="cuda"))
    check_grad(got, ids, dx, vocab, 0.5)
    again = L.embed_backward(ids.int(), dx, vocab, scale=0.5)
    assert torch.equal(got, again)  # a fixed order of additions


def test_gradient_many_tiles_per_block():
    """More keys than 128 blocks of one tile: every block sorts several tiles."""
    n, vocab, I = 2048 * 128 * 2 + 77, 70000, 4
    ids = make_ids(n, vocab, 3, "heavy", torch.int32)
    dx = torch.randn(n, I, device="cuda")
    got = L.embed_backward(ids, dx, vocab)
    ref, mag = expect(ids, dx, vocab, 1.0)
    # sums run over 32 terms, then over units four ways: depth below 32 + n / 128 + 8
    assert bool(((got.double() - ref).abs() <= (40 + n / 128) * 2.0 ** -24 * mag).all())


def test_gradient_accumulates():
    n, vocab, I = 300, 50, 36
    ids = make_ids(n, vocab, 5, "heavy", torch.int64)
    dx = torch.randn(n, I, device="cuda")
    base = torch.randn(vocab, I, device="cuda")
    one = L.embed_backward(ids, dx, vocab, scale=2.0)
    got = L.embed_backward(ids, dx, vocab, scale=2.0, out=base.clone(), accumulate=True)
    touched = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    touched[ids[(ids >= 0) & (ids < vocab)]] = True
    assert torch.equal(got[~touched], base[~touched])
    assert torch.equal(got[touched], (base + one)[touched])


def test_gradient_by_differences():
    """<dtable, E> equals the derivative of <dx, embed(table + t E)> (exact: the lookup is linear)."""
    n, vocab, I, scale = 50, 11, 8, 3.0
    ids = make_ids(n, vocab, 9, "uniform", torch.int64)
    table, E = (torch.randint(-8, 9, (vocab, I), device="cuda").float() for _ in range(2))
    dx = torch.randint(-8, 9, (n, I), device="cuda").float()
    slope = ((L.embed(ids, table + E, scale) - L.embed(ids, table - E, scale)) * dx).double().sum() / 2
    assert float((L.embed_backward(ids, dx, vocab, scale).double() * E).sum()) == float(slope)


def test_empty_and_time_major():
    table = torch.randn(5, 16, device="cuda")
    assert L.embed(torch.empty(0, 3, dtype=torch.int64, device="cuda"), table).shape == (0, 3, 16)
    out = L.embed_backward(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 16, device="cuda"), 5)
    assert torch.equal(out, torch.zeros(5, 16, device="cuda"))
    ids = torch.tensor([[0, 4, 2], [1, -1, 9]], device="cuda")
    x = L.embed(ids, table)
    assert x.shape == (2, 3, 16) and torch.equal(x[0, 1], table[4]) and not x[1, 1:].any()


def test_streams_and_graphs():
    """Two calls at once on two streams with workspaces of their own, and a captured call replayed on new inputs."""
    n, vocab, I = 3000, 400, 64
    ids = make_ids(n, vocab, 1, "heavy", torch.int64)
    dx = torch.randn(n, I, device="cuda")
    want = L.embed_backward(ids, dx, vocab)
    torch.cuda.synchronize()
    ss, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in ss:
        with torch.cuda.stream(s):
            outs.append(L.embed_backward(ids, dx, vocab))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)

    ids_buf, dx_buf, out = torch.zeros_like(ids), torch.zeros_like(dx), torch.empty(vocab, I, device="cuda")
    ws = L.empty_workspace(L.embed_bwd_workspace_size(L.embed_dims(n, vocab, I, torch.float32)), "cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.embed_backward(ids_buf, dx_buf, vocab, out=out, ws=ws)
    ids_buf.copy_(ids)
    dx_buf.copy_(dx)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_ids_from_anywhere():
    ids = torch.arange(9, device="cuda", dtype=torch.int32)
    table = torch.randn(9, 5, device="cuda")
    for r in range(9):
        assert torch.equal(L.embed(ids[r:], table), table[r:])
        assert torch.equal(L.embed_backward(ids[r:], table[r:].contiguous(), 9)[r:], table[r:])


@pytest.mark.parametrize("kind", ["uniform", "same", "heavy"])
@pytest.mark.parametrize("n,vocab", [(4095, 300), (4096, 70000), (4097, 70000), (3000, 262150), (4096, 1)])
def test_gradient_around_the_one_block_sort(n, vocab, kind):
    ids = make_ids(n, vocab, n, kind, torch.int64)
    dx = torch.randn(n, 4, device="cuda")
    got = L.embed_backward(ids, dx, vocab)
    check_grad(got, ids, dx, vocab, 1.0)
    assert torch.equal(got, L.embed_backward(ids, dx, vocab))


def test_sizes_past_an_int():
    ids, table = torch.empty(2 ** 32 + 3, dtype=torch.int32, device="cuda"), torch.zeros(9, 8, device="cuda")
    with pytest.raises(ValueError, match="below 2"):
        L.embed(ids, table)  # (an int would hold 3)
    with pytest.raises(ValueError, match="below 2"):
        L.embed_backward(ids[:5], torch.zeros(5, 8, device="cuda"), 2 ** 32 + 1)


@pytest.mark.parametrize("n", [0, 50, 5000])
@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_gradient_inside_a_buffer(n, at):
    """A table at any element of a buffer: every row is written, nothing beside it is."""
    vocab, I = 777, 5
    buf = torch.full((vocab * I + 8,), 7.0, device="cuda")
    table = buf[at:at + vocab * I].view(vocab, I)
    ids = make_ids(n, vocab, n + at, "heavy", torch.int32)
    dx = torch.randn(n, I, device="cuda")
    got = L.embed_backward(ids, dx, vocab, out=table)
    check_grad(got, ids, dx, vocab, 1.0)
    assert bool((buf[:at] == 7.0).all()) and bool((buf[at + vocab * I:] == 7.0).all())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("I", [1024, 259])
def test_sums_of_a_frequent_token(I, dt):
    """Rows whose sums over any 32 are exact in float: the gradient of a token of 130000 rows is its sum rounded once,
    which chains of float partial sums (2^17 in the end, 2^-18 their digits) are not."""
    n, bits = 131072, {"fp32": 18, "bf16": 7, "fp16": 10}[dt]  # 1 + 5 + 18 bits
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    ids[::1000] = 1
    gen = torch.Generator(device="cuda").manual_seed(I)
    dx = (1 + torch.randint(0, 1 << bits, (n, I), generator=gen, device="cuda").double() / (1 << bits)).to(DT[dt])
    want = torch.stack([dx.double()[ids == w].sum(0) for w in range(3)]).float()
    assert torch.equal(L.embed_backward(ids, dx, 3), want)
    base = torch.randn(3, I, generator=gen, device="cuda")
    assert torch.equal(L.embed_backward(ids, dx, 3, scale=0.5, out=base.clone(), accumulate=True), base + 0.5 * want)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,I", [(3, 8), (3, 7), (70000, 16)])
@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_padding_is_zero_at_any_scale(scale, N, I, dt):
    ids = torch.tensor([-1, 2, 4], device="cuda").repeat(N // 3 + 1)[:N]
    x = L.embed(ids, torch.ones(4, I, device="cuda", dtype=DT[dt]), scale)
    assert not x[ids != 2].any() and not torch.isfinite(x[ids == 2]).any()
