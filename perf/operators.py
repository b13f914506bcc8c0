"""What the gated delta rule, the token embedding and the token log-probabilities of liblstm are measured on.

Three operators of a recurrent language model, each as a user runs it on time-major sequences:

- ``gdr``: the gated delta rule (matrix-state recurrent layer), one forward (serving: single tokens, a few tokens, a
  whole prompt) or a forward and its backward (training);
- ``embed``: rows of an embedding table for token ids, alone (serving) or with the table's gradient (training);
- ``logprob``: log-probability of a given token per row of logits, the row's entropy and its best alternatives, alone
  (scoring, serving) or with the gradient of the logits (training).
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CHUNK = 64


def listed():
    return [
        # one decoding step of 64 sequences: state traffic only
        {"name": "gdr_decode_T1_B64", "op": "gdr", "train": False, "T": 1, "B": 64, "Hk": 8, "Hv": 16, "K": 128, "V": 128, "dtype": "bf16", "ragged": False},
        # a few drafted tokens of a small batch, narrow keys, fp16
        {"name": "gdr_draft_T5_B9_fp16", "op": "gdr", "train": False, "T": 5, "B": 9, "Hk": 4, "Hv": 4, "K": 64, "V": 128, "dtype": "fp16", "ragged": False},
        # one long prompt: few heads, the recurrence over chunks is all there is
        {"name": "gdr_prompt_T8192_B1", "op": "gdr", "train": False, "T": 8192, "B": 1, "Hk": 8, "Hv": 16, "K": 128, "V": 128, "dtype": "bf16", "ragged": False},
        # a training step's layer: enough heads to fill the card
        {"name": "gdr_train_T1024_B16", "op": "gdr", "train": True, "T": 1024, "B": 16, "Hk": 8, "Hv": 16, "K": 128, "V": 128, "dtype": "bf16", "ragged": False},
        # a ragged batch with odd sizes, shared key heads, fp16
        {"name": "gdr_train_ragged_fp16", "op": "gdr", "train": True, "T": 333, "B": 3, "Hk": 2, "Hv": 6, "K": 96, "V": 72, "dtype": "fp16", "ragged": True},
        # the token input of a training step of the benchmark LSTM (T=256, B=128, I=1024)
        {"name": "embed_train_T256_B128", "op": "embed", "train": True, "N": 32768, "vocab": 32000, "I": 1024, "dtype": "bf16", "id64": True},
        # the token input of one decoding step
        {"name": "embed_lookup_B128", "op": "embed", "train": False, "N": 128, "vocab": 32000, "I": 1024, "dtype": "bf16", "id64": True},
        # a small fp32 model over a large vocabulary: most table rows get no gradient
        {"name": "embed_train_odd_fp32", "op": "embed", "train": True, "N": 2049, "vocab": 50001, "I": 260, "dtype": "fp32", "id64": False},
        # the loss of a training step, 8192 rows of logits
        {"name": "logprob_train_N8192", "op": "logprob", "train": True, "N": 8192, "vocab": 32000, "pad": 0, "top": 0, "dtype": "bf16"},
        # scoring with alternatives over a large odd vocabulary in padded rows
        {"name": "logprob_score_N2048", "op": "logprob", "train": False, "N": 2048, "vocab": 100003, "pad": 5, "top": 8, "dtype": "bf16"},
        # one decoding step: few rows, 20 alternatives each
        {"name": "logprob_decode_N4", "op": "logprob", "train": False, "N": 4, "vocab": 128000, "pad": 0, "top": 20, "dtype": "fp32"},
        # a small odd training batch, fp16
        {"name": "logprob_train_odd_fp16", "op": "logprob", "train": True, "N": 117, "vocab": 5001, "pad": 7, "top": 3, "dtype": "fp16"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gdr", "gdr", "embed", "logprob"))
    train = rng.random() < 0.5
    if op == "gdr":
        group = rng.choice((1, 1, 2, 3, 4))
        Hk = _spread(rng, 1, 8)
        B = _spread(rng, 1, 64)
        rows = (1 << 18) // (Hk * group * B)  # T * B * Hv at most that of the training case
        T = _spread(rng, 1, max(1, min(8192, rows)))
        return {"op": "gdr", "train": train, "T": T, "B": B, "Hk": Hk, "Hv": Hk * group, "K": 8 * rng.randint(2, 16), "V": 8 * rng.randint(2, 16),
                "dtype": rng.choice(("bf16", "bf16", "fp16")), "ragged": rng.random() < 0.5}
    if op == "embed":
        I = 4 * _spread(rng, 8, 256)
        return {"op": "embed", "train": train, "N": _spread(rng, 1, 32768), "vocab": _spread(rng, 1000, 32000), "I": I, "dtype": rng.choice(("bf16", "fp16", "fp32")),
                "id64": rng.random() < 0.5}
    vocab = _spread(rng, 1000, 128000)
    return {"op": "logprob", "train": train, "N": _spread(rng, 1, (1 << 27) // vocab), "vocab": vocab, "pad": rng.randint(0, 9), "top": rng.randint(0, 20),
            "dtype": rng.choice(("bf16", "fp16", "fp32"))}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    cd = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    if case["op"] == "gdr":
        T, B, Hk, Hv, K, V = (case[n] for n in ("T", "B", "Hk", "Hv", "K", "V"))
        s = {"q": torch.nn.functional.normalize(randn(T, B, Hk, K), dim=-1).to(cd),
             "k": torch.nn.functional.normalize(randn(T, B, Hk, K), dim=-1).to(cd),
             "v": randn(T, B, Hv, V).to(cd),
             # log decay: minus softplus, most heads remember tens to hundreds of tokens
             "g": -torch.nn.functional.softplus(randn(T, B, Hv) - 3.0),
             "beta": torch.sigmoid(randn(T, B, Hv)),
             "s0": 0.1 * randn(B, Hv, K, V),
             "lengths": None, "scale": K ** -0.5}
        if case["ragged"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            s["lengths"][0] = T
        if case["train"]:
            s["dout"] = randn(T, B, Hv, V).to(cd)
            s["dsT"] = 0.1 * randn(B, Hv, K, V)
    elif case["op"] == "embed":
        N, vocab, I = case["N"], case["vocab"], case["I"]
        # token frequencies fall like 1 / rank; a few positions are padding (-1)
        ids = torch.exp(rand(N) * math.log(vocab)).to(torch.int64).clamp_(1, vocab) - 1
        ids = torch.where(rand(N) < 0.02, torch.full_like(ids, -1), ids)
        s = {"ids": ids if case["id64"] else ids.to(torch.int32), "table": randn(vocab, I).to(cd), "scale": math.sqrt(I)}
        if case["train"]:
            s["dx"] = randn(N, I)
    else:
        N, vocab = case["N"], case["vocab"]
        rows = (3.0 * randn(N, vocab + case["pad"])).to(cd)
        s = {"logits": rows[:, :vocab], "targets": torch.randint(0, vocab, (N,), generator=gen, device=dev), "top": case["top"], "temperature": 0.8}
        if case["train"]:
            s["dlogp"] = -rand(N)
            s["dentropy"] = 0.01 * randn(N)
    s["case"] = dict(case)
    return s


# -------------------------------------------------------------- plain forms
def _gdr_plain(q, k, v, g, beta, s0, lengths, scale):
    """The chunked form in 32 bits: within a chunk the recurrence is a unit lower triangular system."""
    T, B, Hk, K = q.shape
    Hv, V = v.shape[2:]
    pad = -T % CHUNK
    n = (T + pad) // CHUNK
    if lengths is not None:  # a step at or past the length leaves the state alone and gives zeros
        real = (torch.arange(T, device=q.device)[:, None] < lengths[None, :])[:, :, None]
        q, k, v = (torch.where(real[..., None], t, torch.zeros((), device=t.device)) for t in (q, k, v))
        g, beta = (torch.where(real, t, torch.zeros((), device=t.device)) for t in (g, beta))
    q, k = (t.repeat_interleave(Hv // Hk, dim=2) for t in (q, k))
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 0, 0, pad)).reshape(n, CHUNK, B, Hv, -1).permute(0, 2, 3, 1, 4) for t in (q, k, v))
    g, beta = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad)).reshape(n, CHUNK, B, Hv).permute(0, 2, 3, 1) for t in (g, beta))
    b = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    diff = (b[..., :, None] - b[..., None, :]).float()
    gam2 = torch.exp(torch.where(low, diff, torch.zeros_like(diff))) * low
    gam = torch.exp(b.float())[..., None]
    left = torch.exp((b[..., -1:] - b).float())[..., None]
    eye = torch.eye(CHUNK, device=q.device)
    power = -(gam2 * (k @ k.transpose(-1, -2))).tril(-1) * beta[..., None, :]
    inv = eye + power
    for _ in range(5):  # (1 - a)^-1 = (1 + a)(1 + a^2)(1 + a^4)...: a is nilpotent
        power = power @ power
        inv = inv + inv @ power
    p = scale * gam2 * (q @ k.transpose(-1, -2))
    s, out = s0, []
    for c in range(n):
        u = beta[c][..., None] * (inv[c] @ (v[c] - gam[c] * (k[c] @ s)))
        out.append(scale * gam[c] * (q[c] @ s) + p[c] @ u)
        s = gam[c][..., -1:, :] * s + k[c].transpose(-1, -2) @ (left[c] * u)
    o = torch.stack(out).permute(0, 3, 1, 2, 4).reshape(n * CHUNK, B, Hv, V)[:T]
    return o, s


def _plain_gdr(s):
    cd = s["q"].dtype
    names = ("q", "k", "v", "g", "beta", "s0")
    x = {m: s[m].float() for m in names}
    if not s["case"]["train"]:
        o, sT = _gdr_plain(**x, lengths=s["lengths"], scale=s["scale"])
        return {"o": o.to(cd), "sT": sT}
    x = {m: t.detach().requires_grad_() for m, t in x.items()}
    o, sT = _gdr_plain(**x, lengths=s["lengths"], scale=s["scale"])
    grads = torch.autograd.grad((o, sT), [x[m] for m in names], (s["dout"].float(), s["dsT"]))
    res = {"o": o.detach().to(cd), "sT": sT.detach()}
    res.update({"d" + m: t.to(s[m].dtype) for m, t in zip(names, grads)})
    return res


def _plain_embed(s):
    ids, table = s["ids"].long(), s["table"]
    real = (ids >= 0) & (ids < table.shape[0])
    at = torch.where(real, ids, torch.zeros_like(ids))
    x = torch.where(real[:, None], table.float()[at] * s["scale"], torch.zeros((), device=ids.device)).to(table.dtype)
    if not s["case"]["train"]:
        return {"x": x}
    total = torch.zeros(table.shape, dtype=torch.float64, device=ids.device)
    total.index_add_(0, at, torch.where(real[:, None], s["dx"], torch.zeros((), device=ids.device)).double())
    return {"x": x, "dtable": (total * s["scale"]).float()}


def _plain_logprob(s):
    z = s["logits"].float() / s["temperature"]
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    p = e / total
    at = s["targets"].long()[:, None]
    logp = z.gather(1, at) - lse
    entropy = torch.log(total) - (p * (z - top)).sum(1, keepdim=True)
    res = {"logp": logp[:, 0], "entropy": entropy[:, 0]}
    if s["top"]:
        v, i = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        res["top_ids"] = i[:, : s["top"]].to(torch.int32)
        res["top_logp"] = z.gather(1, i[:, : s["top"]]) - lse
    if s["case"]["train"]:
        dz = -s["dlogp"][:, None] * p - s["dentropy"][:, None] * p * (z - lse + entropy)
        dz.scatter_add_(1, at, s["dlogp"][:, None])
        res["dlogits"] = (dz / s["temperature"]).to(s["logits"].dtype)
    return res


# ---------------------------------------------------- the framework's kernels
def _own_gdr(s):
    from backward_lstm_fwd_b200 import binding as L

    train = s["case"]["train"]
    st = L.gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"], lengths=s["lengths"], scale=s["scale"], save=train)
    res = {"o": st.o, "sT": st.sT}
    if train:
        gr = L.gdr_backward(st, s["q"], s["k"], s["v"], s["g"], s["beta"], dout=s["dout"], dsT=s["dsT"], lengths=s["lengths"], scale=s["scale"])
        res.update({"dq": gr.dq, "dk": gr.dk, "dv": gr.dv, "dg": gr.dg, "dbeta": gr.dbeta, "ds0": gr.ds0})
    return res


def _own_embed(s):
    from backward_lstm_fwd_b200 import binding as L

    res = {"x": L.embed(s["ids"], s["table"], scale=s["scale"])}
    if s["case"]["train"]:
        res["dtable"] = L.embed_backward(s["ids"], s["dx"], s["table"].shape[0], scale=s["scale"])
    return res


def _own_logprob(s):
    from backward_lstm_fwd_b200 import binding as L

    st = L.logprobs(s["logits"], s["targets"], top=s["top"], temperature=s["temperature"])
    res = {"logp": st.logp, "entropy": st.entropy}
    if s["top"]:
        res["top_ids"], res["top_logp"] = st.top_ids, st.top_logp
    if s["case"]["train"]:
        res["dlogits"] = L.logprobs_backward(st, s["logits"], s["targets"], dlogp=s["dlogp"], dentropy=s["dentropy"], temperature=s["temperature"])
    return res


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_gdr if op == "gdr" else _own_embed if op == "embed" else _own_logprob)(state)
    return (_plain_gdr if op == "gdr" else _plain_embed if op == "embed" else _plain_logprob)(state)


# ---------------------------------------------------------- 64-bit definition
def _exact_gdr(s):
    """Token by token, the recurrence and its adjoint as the definition writes them."""
    q, k, v, g, beta = (s[m].double() for m in ("q", "k", "v", "g", "beta"))
    T, B, Hk, K = q.shape
    Hv, V = v.shape[2:]
    m = Hv // Hk
    lens = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    live = torch.arange(T, device=q.device)[:, None] < lens[None]
    train = s["case"]["train"]

    def at(t):
        on = live[t][:, None]
        qt, kt = (x[t].repeat_interleave(m, dim=1) * on[..., None] for x in (q, k))
        return qt, kt, v[t] * on[..., None], torch.where(on, torch.exp(g[t]), torch.ones_like(g[t])), beta[t] * on

    def step(S, t):
        qt, kt, vt, a, bt = at(t)
        Sd = a[..., None, None] * S
        r = vt - torch.einsum("bhk,bhkv->bhv", kt, Sd)
        return Sd, r, Sd + kt[..., None] * (bt[..., None] * r)[..., None, :], qt, kt, a, bt

    S = s["s0"].double()
    o = torch.zeros(T, B, Hv, V, dtype=torch.float64, device=q.device)
    marks = {}
    for t in range(T):
        if train and t % 32 == 0:
            marks[t] = S
        _, _, S, qt, *_ = step(S, t)
        o[t] = s["scale"] * torch.einsum("bhk,bhkv->bhv", qt, S)
    res = {"o": o, "sT": S}
    if not train:
        return res
    do = s["dout"].double() * live[:, :, None, None]
    D = s["dsT"].double()
    dq, dk = (torch.zeros(T, B, Hv, K, dtype=torch.float64, device=q.device) for _ in range(2))
    dv, dg, dbeta = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
    for t0 in sorted(marks, reverse=True):
        S, kept = marks[t0], []
        for t in range(t0, min(T, t0 + 32)):
            kept.append(step(S, t))
            S = kept[-1][2]
        for t in range(min(T, t0 + 32) - 1, t0 - 1, -1):
            Sd, r, S1, qt, kt, a, bt = kept[t - t0]
            dq[t] = s["scale"] * torch.einsum("bhkv,bhv->bhk", S1, do[t])
            D = D + s["scale"] * qt[..., None] * do[t][..., None, :]
            du = torch.einsum("bhk,bhkv->bhv", kt, D)
            dbeta[t] = (du * r).sum(-1)
            dr = bt[..., None] * du
            dv[t] = dr
            dk[t] = torch.einsum("bhkv,bhv->bhk", D, bt[..., None] * r) - torch.einsum("bhkv,bhv->bhk", Sd, dr)
            D = D - kt[..., None] * dr[..., None, :]
            dg[t] = (D * Sd).sum((-1, -2))
            D = a[..., None, None] * D
    on = live[:, :, None]
    dq, dk = ((x * on[..., None]).reshape(T, B, Hk, m, K).sum(3) for x in (dq, dk))
    res.update({"dq": dq, "dk": dk, "dv": dv * on[..., None], "dg": dg * on, "dbeta": dbeta * on, "ds0": D})
    return res


def _exact_embed(s):
    table, ids = s["table"].double(), s["ids"].tolist()
    N, (vocab, I) = len(ids), table.shape
    x = torch.zeros(N, I, dtype=torch.float64, device=table.device)
    rows = [r for r, w in enumerate(ids) if 0 <= w < vocab]
    at = torch.tensor(rows, device=table.device, dtype=torch.int64)
    words = torch.tensor([ids[r] for r in rows], device=table.device, dtype=torch.int64)
    x[at] = table[words] * s["scale"]
    res = {"x": x}
    if s["case"]["train"]:
        # rows of equal words side by side, then differences of one running sum per column
        order = torch.argsort(words, stable=True)
        run_sum = torch.cumsum(s["dx"].double()[at[order]], 0)
        ends = torch.cumsum(torch.bincount(words, minlength=vocab), 0)
        run_sum = torch.cat([torch.zeros(1, I, dtype=torch.float64, device=table.device), run_sum])
        upto = run_sum[ends]
        res["dtable"] = s["scale"] * torch.diff(upto, dim=0, prepend=torch.zeros(1, I, dtype=torch.float64, device=table.device))
    return res


def _exact_logprob(s):
    N, parts = s["logits"].shape[0], []
    block = max(1, (1 << 25) // s["logits"].shape[1])
    for r in range(0, N, block):
        z = s["logits"][r:r + block].double() / s["temperature"]
        t = s["targets"][r:r + block].long()
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        p = torch.exp(lp)
        h = -(p * lp).sum(1)
        one = {"logp": lp[torch.arange(len(t), device=t.device), t], "entropy": h}
        if s["top"]:
            # the largest by value, the lowest index first among equals
            i = torch.argsort(-s["logits"][r:r + block].double(), dim=1, stable=True)[:, : s["top"]]
            one["top_ids"], one["top_logp"] = i.to(torch.int32), lp.gather(1, i)
        if s["case"]["train"]:
            hot = torch.zeros_like(p)
            hot[torch.arange(len(t), device=t.device), t] = 1.0
            d = s["dlogp"][r:r + block].double()[:, None] * (hot - p) - s["dentropy"][r:r + block].double()[:, None] * p * (lp + h[:, None])
            one["dlogits"] = d / s["temperature"]
        parts.append(one)
    return {m: torch.cat([x[m] for x in parts]) for m in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gdr":
        return _exact_gdr(s)
    return _exact_embed(s) if case["op"] == "embed" else _exact_logprob(s)


# ------------------------------------------------------------------- floors
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "gdr":
        T, B, Hk, Hv, K, V = (case[n] for n in ("T", "B", "Hk", "Hv", "K", "V"))
        rows = T * B
        qkv = rows * (2 * Hk * K + Hv * V) * e
        gates, state = 2 * rows * Hv * 4, B * Hv * K * V * 4
        bytes_ = qkv + gates + rows * Hv * V * e + 2 * state
        # per token and head: the state's read by k, its rank-one update, its read by q
        flops = rows * Hv * 6.0 * K * V
        if case["train"]:
            bytes_ += 2 * qkv + gates + rows * Hv * V * e + 2 * state + gates
            flops *= 3
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "embed":
        N, vocab, I = case["N"], case["vocab"], case["I"]
        ids = N * (8 if case["id64"] else 4)
        # distinct words among N with frequencies 1 / rank: each table row is read once
        seen = sum(1.0 - math.exp(N * math.log1p(-min(0.999999, math.log((w + 1) / w) / math.log(vocab)))) for w in range(1, vocab))
        bytes_ = ids + (min(seen, N) + N) * I * e
        flops = float(N * I)
        if case["train"]:
            bytes_ += ids + N * I * 4 + vocab * I * 4
            flops += 2.0 * N * I
        return {"bytes": bytes_, "flops": flops}
    N, vocab = case["N"], case["vocab"]
    bytes_ = N * vocab * e + N * 8 + N * 8 + N * case["top"] * 8
    flops = 6.0 * N * vocab
    if case["train"]:
        bytes_ += 2 * N * vocab * e + N * 16
        flops += 8.0 * N * vocab
    return {"bytes": bytes_, "flops": flops}
