"""The router's balance loss, the router gate's gradient and the low-rank
adapters beside a projection: measured cases, inputs and plain forms.

Three operators, told apart by a case's "op":

``balance``   per-expert counts and the sequence-wise balance loss of a sigmoid
              router: over the valid tokens t of a sequence q,
              p_te = s_te / sum_e s_te with s = sigmoid(logits),
              counts_qe = routing entries of q to expert e,
              loss = coeff / Q' * sum_q E / (k n_q^2) * sum_e counts_qe P_qe,
              P_qe = sum_t p_te, n_q the valid tokens of q and Q' the sequences
              that have one.
``gate_grad`` the gradient of the logits, from the gradient of the gate's
              weights w_j = s_j / sum_i s_i over a token's picks and from the
              balance loss (its counts are held constant).
``lora``      out_t = base_t + scale_a (x_t A_a^T) B_a^T with a the adapter of
              token t's request; a token without one keeps its row.
"""
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decode batch of the router (128 tokens, 256 experts): launch latency
        {"name": "balance decode", "op": "balance", "T": 128, "E": 256, "k": 8, "Q": 1, "masked": 0.02},
        # a prefill batch of several requests with padding tokens
        {"name": "balance prefill", "op": "balance", "T": 8192, "E": 256, "k": 8, "Q": 5, "masked": 0.05},
        # many picks per token: the counts weigh as much as the probabilities
        {"name": "balance wide top-k", "op": "balance", "T": 65536, "E": 512, "k": 22, "Q": 17, "masked": 0.05},
        # the largest expert count, one global batch
        {"name": "balance large E", "op": "balance", "T": 32768, "E": 2560, "k": 8, "Q": 1, "masked": 0.05},
        # the gradients of the same batches
        {"name": "gate grad decode", "op": "gate_grad", "T": 128, "E": 256, "k": 8, "Q": 1, "masked": 0.02},
        {"name": "gate grad prefill", "op": "gate_grad", "T": 8192, "E": 256, "k": 8, "Q": 5, "masked": 0.05},
        {"name": "gate grad wide top-k", "op": "gate_grad", "T": 65536, "E": 512, "k": 22, "Q": 17, "masked": 0.05},
        {"name": "gate grad large E", "op": "gate_grad", "T": 32768, "E": 2560, "k": 8, "Q": 1, "masked": 0.05},
        # one token of one request beside the router projection (FP32 logits)
        {"name": "lora one token", "op": "lora", "T": 1, "H": 8192, "N": 256, "R": 16, "L": 8, "bf16": False,
         "mix": "tokens"},
        # a decode batch: every token of another request, beside a BF16 projection
        {"name": "lora decode", "op": "lora", "T": 128, "H": 8192, "N": 8192, "R": 16, "L": 32, "bf16": True,
         "mix": "tokens"},
        # prefill beside the router projection: x is read, few columns come out
        {"name": "lora prefill router", "op": "lora", "T": 8192, "H": 8192, "N": 256, "R": 32, "L": 4, "bf16": False,
         "mix": "requests"},
        # prefill of ragged requests beside a square BF16 projection: the largest traffic
        {"name": "lora prefill", "op": "lora", "T": 8192, "H": 8192, "N": 8192, "R": 64, "L": 8, "bf16": True,
         "mix": "requests"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("balance", "gate_grad", "lora"))
    if op != "lora":
        E = _log(rng, 8, 2560)                      # odd counts among them
        T = _log(rng, 1, min(65536, 32768 * 2560 // E))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(22, E)), "Q": rng.randint(1, min(24, T)),
                "masked": rng.choice((0.0, 0.05, 0.3))}
    R = rng.choice((8, 16, 24, 32, 40, 64, 96, 128))
    H, N = 8 * _log(rng, 32, 1024), 8 * _log(rng, 2, 1024)
    L = _log(rng, 1, min(48, 1024 // R))
    T = _log(rng, 1, min(8192, 8192 * 16384 * 512 // ((H + N) * R * L)))
    return {"op": "lora", "T": T, "H": H, "N": N, "R": R, "L": L, "bf16": rng.random() < 0.5,
            "mix": rng.choice(("tokens", "requests"))}


def _cuts(n, parts, g):
    """`parts` ragged pieces of n tokens, as their `parts` + 1 borders (a piece may be empty)."""
    inner = torch.sort(torch.randint(0, n + 1, (parts - 1,), generator=g)).values
    return torch.cat([torch.zeros(1, dtype=torch.int64), inner, torch.full((1,), n)])


def _prepare_router(c, seed):
    T, E, k, Q = c["T"], c["E"], c["k"], c["Q"]
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    logits = 1.5 * torch.randn(T, E, generator=gd, device=DEV) + 0.7 * torch.randn(E, generator=gd, device=DEV)
    valid = torch.rand(T, generator=gd, device=DEV) >= c["masked"]
    bias = 0.1 * torch.rand(E, generator=gd, device=DEV)
    ids = torch.topk(torch.sigmoid(logits) + bias, k, dim=1).indices.to(torch.int32)
    ids[~valid] = -1
    logits[~valid] = float("nan")                   # padding: never read
    s = {"case": c, "logits": logits, "ids": ids, "mask": valid.to(torch.uint8), "coeff": 1e-2,
         "offsets": None if Q == 1 else _cuts(T, Q, g).to(torch.int32).to(DEV)}
    if c["op"] == "gate_grad":                      # what the forward pass left, and the gradients that arrive
        s["grad_w"] = torch.randn(T, k, generator=gd, device=DEV)
        s["grad_loss"] = 0.5 + torch.rand(1, generator=gd, device=DEV)
        seq = _sequence_of(s)
        live = valid & (seq < Q)
        s["seq_tokens"] = torch.zeros(Q + 1, dtype=torch.int32, device=DEV).scatter_add_(
            0, seq, live.to(torch.int32))[:Q].contiguous()
        s["counts"] = _counts(s, seq, live)
    return s


def _prepare_lora(c, seed):
    T, H, N, R, L = c["T"], c["H"], c["N"], c["R"], c["L"]
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    if c["mix"] == "tokens":                        # decode: each token is another request's; some carry none
        ids = torch.randint(0, L, (T,), generator=g)
        ids[torch.rand(T, generator=g) < 0.06] = -1
    else:                                           # prefill: requests one after the other, some with no adapter
        parts = min(T, max(2, L + L // 2))
        cuts = _cuts(T, parts, g)
        of = torch.randint(-1, L, (parts,), generator=g)
        ids = of[torch.searchsorted(cuts[1:-1].contiguous(), torch.arange(T), right=True)]
    if T == 1:
        ids[0] = seed % L
    out_type = torch.bfloat16 if c["bf16"] else torch.float32
    rnd = lambda *shape: torch.randn(*shape, generator=gd, device=DEV)  # noqa: E731
    return {"case": c, "x": rnd(T, H).to(torch.bfloat16), "base": rnd(T, N).to(out_type),
            "a": (rnd(L, R, H) * H ** -0.5).to(torch.bfloat16), "b": (rnd(L, N, R) * (0.5 * R ** -0.5)).to(torch.bfloat16),
            "scales": 0.5 + 1.5 * torch.rand(L, generator=gd, device=DEV), "ids": ids.to(torch.int32).to(DEV)}


def prepare(case, seed):
    return _prepare_lora(case, seed) if case["op"] == "lora" else _prepare_router(case, seed)


# ---------------------------------------------------------------------- plain forms
def _sequence_of(s):
    """The sequence of each token (Q: of none)."""
    T, Q = s["case"]["T"], s["case"]["Q"]
    if s["offsets"] is None:
        return torch.zeros(T, dtype=torch.int64, device=DEV)
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    return torch.searchsorted(s["offsets"][1:].contiguous(), t, right=True).clamp(max=Q)


def _counts(s, seq, live):
    E, Q = s["case"]["E"], s["case"]["Q"]
    ids = s["ids"].long()
    ok = live[:, None] & (ids >= 0) & (ids < E)
    flat = torch.where(ok, seq[:, None] * E + ids, Q * E)
    hist = torch.zeros(Q * E + 1, dtype=torch.int32, device=DEV)
    hist.scatter_add_(0, flat.reshape(-1), torch.ones(flat.numel(), dtype=torch.int32, device=DEV))
    return hist[:-1].view(Q, E).contiguous()


def _plain_balance(s):
    c = s["case"]
    seq = _sequence_of(s)
    live = (s["mask"] != 0) & (seq < c["Q"])
    sig = torch.sigmoid(torch.where(live[:, None], s["logits"], 0.0))
    p = sig / sig.sum(1, keepdim=True)
    member = ((seq[None] == torch.arange(c["Q"], device=DEV)[:, None]) & live[None]).to(torch.float32)
    prob_sums = member @ p
    n = member.sum(1)
    counts = _counts(s, seq, live)
    per = torch.where(n > 0, (counts * prob_sums).sum(1) * c["E"] / (c["k"] * n.clamp(min=1) ** 2), 0.0)
    loss = s["coeff"] * per.sum() / (n > 0).sum().clamp(min=1)
    return {"loss": loss.reshape(1), "counts": counts, "prob_sums": prob_sums, "seq_tokens": n.to(torch.int32)}


def _plain_gate_grad(s):
    c = s["case"]
    E, k, Q = c["E"], c["k"], c["Q"]
    seq = _sequence_of(s)
    valid = s["mask"] != 0
    sig = torch.sigmoid(torch.where(valid[:, None], s["logits"], 0.0))
    total = sig.sum(1, keepdim=True)
    n = s["seq_tokens"].to(torch.float32)
    per = torch.where(n > 0, s["grad_loss"] * s["coeff"] * E / (k * n.clamp(min=1) ** 2), 0.0)
    g = s["counts"] * (per / (n > 0).sum().clamp(min=1))[:, None]
    g = torch.cat([g, torch.zeros(1, E, device=DEV)])[torch.where(valid, seq, Q)]
    grad = (g - (g * sig).sum(1, keepdim=True) / total) * sig * (1 - sig) / total
    ids = s["ids"].long()
    ok = valid[:, None] & (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    sj = sig.gather(1, at) * ok
    w = sj / sj.sum(1, keepdim=True).clamp(min=1e-30)
    dw = torch.where(ok, s["grad_w"], 0.0)
    return grad.scatter_add(1, at, w * (1 - sj) * (dw - (dw * w).sum(1, keepdim=True)))


def _plain_lora(s):
    """Every adapter's product, and each token's own picked out of them."""
    c = s["case"]
    T, H, N, R, L = c["T"], c["H"], c["N"], c["R"], c["L"]
    v = (s["x"].float() @ s["a"].float().view(L * R, H).T).view(T, L, R)
    mine = (s["ids"][:, None] == torch.arange(L, device=DEV)[None]).float() * s["scales"]
    b = s["b"].float().permute(0, 2, 1).reshape(L * R, N)
    return (s["base"].float() + (v * mine[:, :, None]).view(T, L * R) @ b).to(s["base"].dtype)


# ---------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import expert_combine_b200 as eb
        if op == "balance":
            loss, counts, prob_sums, seq_tokens = eb.moe_balance_loss(
                state["logits"], state["ids"], state["mask"], state["coeff"], seq_offsets=state["offsets"])
            return {"loss": loss, "counts": counts, "prob_sums": prob_sums, "seq_tokens": seq_tokens}
        if op == "gate_grad":
            return eb.moe_route_backward(state["logits"], state["ids"], state["mask"], grad_weights=state["grad_w"],
                                         grad_loss=state["grad_loss"], coeff=state["coeff"], counts=state["counts"],
                                         seq_tokens=state["seq_tokens"], seq_offsets=state["offsets"])
        return eb.lora_add(state["base"], state["x"], state["a"], state["b"], state["ids"], scales=state["scales"])
    return {"balance": _plain_balance, "gate_grad": _plain_gate_grad, "lora": _plain_lora}[op](state)


def work(case):
    c = case
    if c["op"] == "lora":
        used = min(c["L"], c["T"])
        size = 2 if c["bf16"] else 4
        return {"bytes": c["T"] * (2 * c["H"] + 2 * size * c["N"] + 4) + 2 * used * c["R"] * (c["H"] + c["N"]),
                "flops": 2 * c["T"] * c["R"] * (c["H"] + c["N"])}
    TE, Tk = c["T"] * c["E"], c["T"] * c["k"]
    if c["op"] == "balance":
        return {"bytes": 4 * TE + 4 * Tk + c["T"] + 8 * c["Q"] * c["E"], "flops": 6 * TE}
    return {"bytes": 8 * TE + 8 * Tk + c["T"] + 4 * c["Q"] * c["E"], "flops": 10 * TE}


# ---------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The router's operators sequence by sequence, the adapters one by one, from the definitions in 64 bits."""
    s, c, f = prepare(case, seed), case, torch.float64
    if c["op"] == "lora":
        out = s["base"].to(f)
        for a in range(c["L"]):
            t = torch.nonzero(s["ids"] == a).flatten()
            if len(t):
                v = s["x"][t].to(f) @ s["a"][a].to(f).T
                out[t] += s["scales"][a].to(f) * (v @ s["b"][a].to(f).T)
        return out
    T, E, k, Q = c["T"], c["E"], c["k"], c["Q"]
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    counts, probs = torch.zeros(Q, E, dtype=f, device=DEV), torch.zeros(Q, E, dtype=f, device=DEV)
    rows = []
    for q in range(Q):
        t = torch.arange(cuts[q], cuts[q + 1], device=DEV)
        t = t[s["mask"][t] != 0]
        rows.append(t)
        if len(t):
            p = 1 / (1 + torch.exp(-s["logits"][t].to(f)))
            probs[q] = (p / p.sum(1, keepdim=True)).sum(0)
            picks = s["ids"][t].reshape(-1)
            counts[q] = torch.bincount(picks[picks >= 0].long(), minlength=E).to(f)
    some = max(1, sum(len(t) > 0 for t in rows))
    if c["op"] == "balance":
        loss = sum(float((counts[q] * probs[q]).sum()) * E / (k * len(t) ** 2) for q, t in enumerate(rows) if len(t))
        return {"loss": torch.tensor([s["coeff"] * loss / some], dtype=f), "counts": counts.to(torch.int32),
                "prob_sums": probs, "seq_tokens": torch.tensor([len(t) for t in rows], dtype=torch.int32)}
    grad = torch.zeros(T, E, dtype=f, device=DEV)
    for q, t in enumerate(rows):
        if not len(t):
            continue
        x = s["logits"][t].to(f)
        p = 1 / (1 + torch.exp(-x))
        slope = p / (1 + torch.exp(x))
        g = float(s["grad_loss"].to(f)) * s["coeff"] * E / (some * k * len(t) ** 2) * counts[q]
        S = p.sum(1, keepdim=True)
        d = slope * (g / S - (p @ g)[:, None] / S ** 2)
        at = s["ids"][t].long()
        sj = p.gather(1, at)
        W = sj.sum(1, keepdim=True)
        dw = s["grad_w"][t].to(f)
        d.scatter_add_(1, at, slope.gather(1, at) * (dw / W - (dw * sj).sum(1, keepdim=True) / W ** 2))
        grad[t] = d
    return grad
