"""The boundary of the embedding and log-probability entry points, checked
without a GPU: every rejected call returns before its first CUDA call."""
import ctypes

import pytest
import torch

from backward_lstm_fwd_b200 import binding as L
from backward_lstm_fwd_b200 import build as lbuild

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return L.load()


# ---------------------------------------------------------------- embedding
def embed_fwd(lib, d, ids=FAKE, table=FAKE, x=FAKE):
    return lib.lstm_embed_fwd(ctypes.byref(d), ids, table, 1.0, x, None)


def embed_bwd(lib, d, ids=FAKE, dx=FAKE, dtable=FAKE, ws=FAKE, ws_bytes=None, accumulate=0):
    n = L.embed_bwd_workspace_size(d) if ws_bytes is None else ws_bytes
    return lib.lstm_embed_bwd(ctypes.byref(d), ids, dx, 1.0, accumulate, dtable, ws, n, None)


@pytest.mark.parametrize("bad", [(-1, 5, 8, 0, 8), (4, -5, 8, 0, 8), (4, 5, -8, 0, 8), (4, 5, 8, 3, 8), (4, 5, 8, 0, 2)])
def test_embed_dims(lib, bad):
    d = L.embed_dims(*bad[:3], bad[3], bad[4])
    assert embed_fwd(lib, d) == L.LSTM_ERR_INVALID_ARG
    assert embed_bwd(lib, d, ws_bytes=1 << 30) == L.LSTM_ERR_INVALID_ARG
    assert L.embed_bwd_workspace_size(d) == 0


def test_embed_pointers_and_workspace(lib):
    d = L.embed_dims(4, 5, 8, L.LSTM_BF16)
    for k in ("ids", "table", "x"):
        assert embed_fwd(lib, d, **{k: None}) == L.LSTM_ERR_INVALID_ARG
        assert embed_fwd(lib, d, **{k: FAKE + 1}) == L.LSTM_ERR_INVALID_ARG
    for k in ("ids", "dx", "dtable"):
        assert embed_bwd(lib, d, **{k: None}) == L.LSTM_ERR_INVALID_ARG
        assert embed_bwd(lib, d, **{k: FAKE + 1}) == L.LSTM_ERR_INVALID_ARG
    assert embed_fwd(lib, d, ids=FAKE + 4) == L.LSTM_ERR_INVALID_ARG  # ids of 8 bytes
    assert embed_bwd(lib, d, accumulate=2) == L.LSTM_ERR_INVALID_ARG
    need = L.embed_bwd_workspace_size(d)
    assert embed_bwd(lib, d, ws_bytes=need - 1) == L.LSTM_ERR_WORKSPACE
    assert embed_bwd(lib, d, ws=None) == L.LSTM_ERR_WORKSPACE
    assert embed_bwd(lib, d, ws=FAKE + 16) == L.LSTM_ERR_WORKSPACE
    assert lib.lstm_embed_fwd(None, FAKE, FAKE, 1.0, FAKE, None) == L.LSTM_ERR_INVALID_ARG
    # nothing to do: nothing is enqueued
    assert embed_fwd(lib, L.embed_dims(0, 5, 8, 0), ids=None, x=None) == L.LSTM_OK
    assert embed_bwd(lib, L.embed_dims(4, 0, 8, 0), dtable=None) == L.LSTM_OK


def test_embed_extents(lib):
    assert embed_fwd(lib, L.embed_dims(4, (1 << 30) + 1, 8, 0)) == L.LSTM_ERR_UNSUPPORTED
    assert embed_bwd(lib, L.embed_dims(4, 5, (1 << 24) + 1, 0), ws_bytes=1 << 40) == L.LSTM_ERR_UNSUPPORTED


# --------------------------------------------------------- log-probabilities
def logprob_fwd(lib, d, inv_temp=1.0, logits=FAKE, targets=FAKE, logp=FAKE, entropy=FAKE, stats=FAKE, top_ids=FAKE,
                top_logp=FAKE):
    return lib.lstm_logprob_fwd(ctypes.byref(d), logits, targets, inv_temp, logp, entropy, stats, top_ids, top_logp,
                                None)


def logprob_bwd(lib, d, inv_temp=1.0, logits=FAKE, targets=FAKE, stats=FAKE, entropy=FAKE, dlogp=FAKE, dentropy=FAKE,
                dlogits=2 * FAKE, ldd=None):
    return lib.lstm_logprob_bwd(ctypes.byref(d), logits, targets, inv_temp, stats, entropy, dlogp, dentropy, dlogits,
                                d.vocab if ldd is None else ldd, None)


@pytest.mark.parametrize("kw", [dict(N=-1, vocab=9), dict(N=2, vocab=-1), dict(N=2, vocab=9, ld=8), dict(N=2, vocab=9, top=10),
                                dict(N=2, vocab=9, top=-1), dict(N=2, vocab=9, dtype=5), dict(N=2, vocab=9, id_bytes=1)])
def test_logprob_dims(lib, kw):
    kw.setdefault("dtype", L.LSTM_F32)
    d = L.logprob_dims(**kw)
    assert logprob_fwd(lib, d) == L.LSTM_ERR_INVALID_ARG
    assert logprob_bwd(lib, d) == L.LSTM_ERR_INVALID_ARG


def test_logprob_arguments(lib):
    d = L.logprob_dims(3, 100, L.LSTM_F16, top=4)
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-30):
        assert logprob_fwd(lib, d, inv_temp=t) == L.LSTM_ERR_INVALID_ARG
        assert logprob_bwd(lib, d, inv_temp=t) == L.LSTM_ERR_INVALID_ARG
    for k in ("logits", "targets", "stats", "top_ids", "top_logp"):
        assert logprob_fwd(lib, d, **{k: None}) == L.LSTM_ERR_INVALID_ARG
    for k in ("logits", "targets", "logp", "entropy", "stats", "top_ids", "top_logp"):
        assert logprob_fwd(lib, d, **{k: FAKE + 1}) == L.LSTM_ERR_INVALID_ARG
    assert logprob_fwd(lib, d, targets=FAKE + 4) == L.LSTM_ERR_INVALID_ARG
    for k in ("logits", "targets", "stats", "entropy", "dlogits"):
        assert logprob_bwd(lib, d, **{k: None}) == L.LSTM_ERR_INVALID_ARG
        assert logprob_bwd(lib, d, **{k: FAKE + 1}) == L.LSTM_ERR_INVALID_ARG
    assert logprob_bwd(lib, d, ldd=99) == L.LSTM_ERR_INVALID_ARG
    assert logprob_bwd(lib, d, dlogits=FAKE, ldd=104) == L.LSTM_ERR_INVALID_ARG  # in place with another stride
    assert logprob_fwd(lib, L.logprob_dims(3, 100, 0, top=65)) == L.LSTM_ERR_UNSUPPORTED
    # nothing to do: nothing is enqueued
    assert logprob_fwd(lib, L.logprob_dims(0, 100, 0, top=4), logits=None, targets=None, logp=None, stats=None, top_ids=None,
                       top_logp=None) == L.LSTM_OK
    assert logprob_bwd(lib, L.logprob_dims(0, 100, 0), dlogits=None) == L.LSTM_OK


def test_binding_refuses_host_tensors_and_shapes(lib):
    ids, table = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        L.embed(ids, table)
    with pytest.raises(ValueError, match="CUDA"):
        L.embed_backward(ids, torch.zeros(3, 8), 5)
    with pytest.raises(ValueError, match="CUDA"):
        L.logprobs(torch.zeros(3, 5), ids)
    with pytest.raises(ValueError, match="below 2"):
        L.logprobs(torch.empty(1, 2 ** 31 + 5, device="meta"))  # (an int would hold 5)
    with pytest.raises(ValueError, match="rows overlap"):
        L.logprobs(torch.zeros(1, 5).expand(3, 5), ids)
    with pytest.raises(ValueError, match="dense"):
        L.logprobs(torch.zeros(5, 3).t(), ids)


# ----------------------------------------------------------- gated delta rule
def gdr_fwd(lib, d, opt=None, q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, s0=None, o=FAKE, sT=FAKE, states=None, deltas=None,
            ws=FAKE, ws_bytes=None):
    n = L.gdr_fwd_workspace_size(d, states is not None) if ws_bytes is None else ws_bytes
    return lib.lstm_gdr_fwd(ctypes.byref(d), ctypes.byref(opt) if opt else None, q, k, v, g, beta, s0, o, sT, states, deltas,
                            ws, n, None)


def gdr_bwd(lib, d, opt=None, dout=FAKE, dsT=FAKE, q=FAKE, k=FAKE, v=None, g=FAKE, beta=FAKE, states=FAKE, deltas=FAKE, dq=FAKE,
            dk=FAKE, dv=FAKE, dg=FAKE, dbeta=FAKE, ds0=FAKE, fwd_ws=None, ws=FAKE, ws_bytes=None):
    n = L.gdr_bwd_workspace_size(d) if ws_bytes is None else ws_bytes
    return lib.lstm_gdr_bwd(ctypes.byref(d), ctypes.byref(opt) if opt else None, dout, dsT, q, k, v, g, beta, states, deltas,
                            dq, dk, dv, dg, dbeta, ds0, fwd_ws, ws, n, None)


GDR = dict(T=100, B=2, Hk=2, Hv=4, K=64, V=64, dtype=L.LSTM_BF16)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(B=-1), dict(Hk=-1), dict(Hv=-2), dict(K=-8), dict(V=-8), dict(dtype=3),
                                 dict(Hv=3), dict(Hk=0), dict(ldq=64), dict(ldk=64), dict(ldv=64), dict(T=1 << 20, B=1 << 12)])
def test_gdr_dims(lib, bad):
    d = L.gdr_dims(**{**GDR, **bad})
    assert gdr_fwd(lib, d, ws_bytes=1 << 40) == L.LSTM_ERR_INVALID_ARG
    assert gdr_bwd(lib, d, ws_bytes=1 << 40) == L.LSTM_ERR_INVALID_ARG
    assert L.gdr_fwd_workspace_size(d) == 0 == L.gdr_bwd_workspace_size(d)


@pytest.mark.parametrize("big", [dict(K=136), dict(V=264), dict(K=60), dict(V=60), dict(ldq=132), dict(ldv=260)])
def test_gdr_extents(lib, big):
    d = L.gdr_dims(**{**GDR, **big})
    assert gdr_fwd(lib, d, ws_bytes=1 << 40) == L.LSTM_ERR_UNSUPPORTED
    assert gdr_bwd(lib, d, ws_bytes=1 << 40) == L.LSTM_ERR_UNSUPPORTED
    assert L.gdr_fwd_workspace_size(d) == 0 == L.gdr_bwd_workspace_size(d)


def test_gdr_arguments(lib):
    d = L.gdr_dims(**GDR)
    by_element = ("g", "beta", "dg", "dbeta")
    for n in ("q", "k", "v", "g", "beta", "o", "sT"):
        assert gdr_fwd(lib, d, **{n: None}) == L.LSTM_ERR_INVALID_ARG
        assert gdr_fwd(lib, d, **{n: FAKE + (2 if n in by_element else 8)}) == L.LSTM_ERR_INVALID_ARG
    assert gdr_fwd(lib, d, s0=FAKE + 8) == L.LSTM_ERR_INVALID_ARG
    assert gdr_fwd(lib, d, states=FAKE) == L.LSTM_ERR_INVALID_ARG  # the backward needs both
    assert gdr_fwd(lib, d, deltas=FAKE) == L.LSTM_ERR_INVALID_ARG
    for n in ("q", "k", "g", "beta", "states", "deltas", "dq", "dk", "dv", "dg", "dbeta"):
        assert gdr_bwd(lib, d, **{n: None}) == L.LSTM_ERR_INVALID_ARG
        assert gdr_bwd(lib, d, **{n: FAKE + (2 if n in by_element else 8)}) == L.LSTM_ERR_INVALID_ARG
    assert gdr_bwd(lib, d, fwd_ws=FAKE + 16) == L.LSTM_ERR_INVALID_ARG
    for opt in (L.GdrOptions(FAKE + 2, 1.0), L.GdrOptions(None, float("nan")), L.GdrOptions(None, float("inf"))):
        assert gdr_fwd(lib, d, opt=opt) == L.LSTM_ERR_INVALID_ARG
        assert gdr_bwd(lib, d, opt=opt) == L.LSTM_ERR_INVALID_ARG
    for save in (None, FAKE):
        need = L.gdr_fwd_workspace_size(d, save is not None)
        assert need > 256
        assert gdr_fwd(lib, d, states=save, deltas=save, ws_bytes=need - 1) == L.LSTM_ERR_WORKSPACE
        assert gdr_fwd(lib, d, states=save, deltas=save, ws=None) == L.LSTM_ERR_WORKSPACE
    assert gdr_bwd(lib, d, ws_bytes=L.gdr_bwd_workspace_size(d) - 1) == L.LSTM_ERR_WORKSPACE
    # a few tokens that keep nothing need the control block alone
    few = L.gdr_dims(**{**GDR, "T": 1})
    assert L.gdr_fwd_workspace_size(few) == 256 < L.gdr_fwd_workspace_size(few, True)
    assert gdr_fwd(lib, few, ws=FAKE + 16) == L.LSTM_ERR_WORKSPACE  # (NULL would do, this not)
    assert gdr_fwd(lib, few, ws=FAKE, ws_bytes=255) == L.LSTM_ERR_WORKSPACE
    assert gdr_fwd(lib, few, states=FAKE, deltas=FAKE, ws=None) == L.LSTM_ERR_WORKSPACE
    # nothing to do: nothing is enqueued
    none = L.gdr_dims(**{**GDR, "B": 0})
    assert gdr_fwd(lib, none, q=None, k=None, v=None, g=None, beta=None, o=None, sT=None) == L.LSTM_OK
    assert gdr_bwd(lib, none) == L.LSTM_OK


def test_gdr_lengths_past_an_int(lib):
    d = L.gdr_dims(2 ** 31 - 1, 1, 1, 1, 8, 8, torch.bfloat16)  # (its chunks' count would wrap)
    assert gdr_fwd(lib, d, ws_bytes=1 << 60) == L.LSTM_ERR_UNSUPPORTED
    assert gdr_bwd(lib, d, ws_bytes=1 << 60) == L.LSTM_ERR_UNSUPPORTED


def test_gdr_binding_refusals(lib):
    q = torch.zeros(4, 2, 1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        L.gdr_forward(q, q, q, torch.zeros(4, 2, 1), torch.zeros(4, 2, 1))
    with pytest.raises(ValueError, match="heads must be dense"):
        L._token_stride(torch.zeros(4, 2, 2, 16)[..., :8], "q")
    with pytest.raises(ValueError, match="one stride"):
        L._token_stride(torch.zeros(4, 3, 1, 8)[:, :2], "q")
    assert L._token_stride(torch.zeros(4, 2, 24)[..., 8:16].view(4, 2, 1, 8), "q") == 24
