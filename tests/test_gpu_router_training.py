"""Balance loss and gate gradient on the GPU against their definitions in
binary64.

Tolerances, in units u = 2^-24 (half a step of binary32, relative).  A sigmoid
costs: its exponent's product, |x| u; 2^x and the reciprocal, 2 steps = 4 u and
1 step = 2 u; the addition, u.  A row's sum of E positive terms adds at most
16 + 5 + 8 roundings (lane, butterfly, warps), its reciprocal and product 3.
So a probability is off by at most (max|x| + 40) u.  A token range is summed in
64 + 8 steps, the slots of a sequence in T / (16 * 8) + 16 at most.
"""
import numpy as np
import pytest
import torch

import expert_combine_b200 as eb
from router_training import backward, balance

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(T, E, k, seed, masked=0.2, scale=2.0, shift=0.0):
    r = np.random.default_rng(seed)
    x = (r.normal(size=(T, E)) * scale + shift).astype(np.float32)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = (r.random(T) >= masked).astype(np.uint8)
    x[mask == 0] = np.nan                               # never used
    dw = r.normal(size=(T, k)).astype(np.float32)
    return x, ids, mask, dw


def _dev(dev, *arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def _xmax(x):
    v = np.abs(x[np.isfinite(x)])
    return float(v.max()) if v.size else 0.0


def _check(dev, x, ids, mask, dw, off=None, coeff=0.3, grad_loss=1.25):
    T, E = x.shape
    tx, ti, tm, tw, to = _dev(dev, x, ids, mask, dw, None if off is None else np.asarray(off, np.int32))
    loss, counts, probs, n = eb.moe_balance_loss(tx, ti, tm, coeff, seq_offsets=to)
    gl = torch.tensor([grad_loss], device=dev)
    both = eb.moe_route_backward(tx, ti, tm, grad_weights=tw, grad_loss=gl, coeff=coeff, counts=counts, seq_tokens=n,
                                 seq_offsets=to)
    gate = eb.moe_route_backward(tx, ti, tm, grad_weights=tw)
    bal = eb.moe_route_backward(tx, ti, tm, grad_loss=gl, coeff=coeff, counts=counts, seq_tokens=n, seq_offsets=to)
    torch.cuda.synchronize()
    rl, rc, rp, rn = balance(x, ids, mask, coeff, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(n.cpu().numpy(), rn)
    each = _xmax(x[mask != 0]) + 40
    tol = (each + 72 + T / 128 + 16) * U
    assert np.all(np.abs(probs.cpu().numpy() - rp) <= tol * rp + 1e-37)
    # the loss: a tree of at most 5 + E / 32 + Q additions more, and 8 operations
    assert abs(float(loss) - rl) <= (tol + (5 + E / 32 + len(rn) + 8) * U) * abs(rl)
    # a gradient: each of g - G's two terms, the slope (2 products, sum's reciprocal) and the gate's part
    for got, want in ((both, dict(grad_w=dw, grad_loss=grad_loss)), (gate, dict(grad_w=dw)),
                      (bal, dict(grad_loss=grad_loss))):
        rg, mag = backward(x, ids, mask, coeff=coeff, counts=rc, seq_tokens=rn, offsets=off, **want)
        err = np.abs(got.cpu().numpy() - rg)
        assert np.all(err <= (2 * each + 60) * U * mag + 1e-37), float((err / (mag + 1e-37)).max() / U)
        assert not got.cpu().numpy()[mask == 0].any()


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (1, 256, 8), (2, 9, 9), (127, 37, 5), (64, 64, 32), (300, 128, 6),
                                   (129, 256, 8), (65, 257, 8), (40, 512, 22), (33, 513, 3), (50, 1000, 8),
                                   (20, 1500, 8), (21, 2560, 8), (9, 3001, 4), (10, 4096, 32)])
def test_sizes(cuda_dev, T, E, k):
    _check(cuda_dev, *_inputs(T, E, k, seed=T + E))


@pytest.mark.parametrize("off", [[0, 100], [0, 0, 1, 1, 50, 100, 100], [7, 9, 60, 90], [100, 100], [0, 0],
                                 list(range(101)), [0, 33, 34, 99]])
def test_sequences(cuda_dev, off):
    """Empty sequences, single tokens, tokens in front of the first and behind the last."""
    _check(cuda_dev, *_inputs(100, 48, 4, seed=len(off)), off=off)


def test_long_batches_cut_anywhere(cuda_dev):
    """More tokens than one CTA's range holds, borders inside the ranges."""
    x, ids, mask, dw = _inputs(6000, 16, 2, seed=3)
    _check(cuda_dev, x, ids, mask, dw, off=[0, 1, 17, 2049, 2050, 5999, 6000])
    _check(cuda_dev, x[:, :9], np.clip(ids, -1, 9), mask, dw)    # id 9: outside E = 9


@pytest.mark.parametrize("T,E,k,off", [(5000, 64, 6, [0, 1, 1, 40, 41, 2500, 4990]), (5001, 66, 6, [3, 2049, 5001]),
                                       (300, 1000, 8, [0, 17, 150, 299]), (130, 2560, 8, [1, 64, 65, 130]),
                                       (90, 4096, 32, None), (88, 3001, 8, [0, 44, 88]), (40, 2560, 4, [0, 7, 8, 40]),
                                       (600, 512, 22, None)])
def test_batches_of_many_ctas(cuda_dev, T, E, k, off):
    """Sums that pass through slots of several CTAs, or more sums than a cluster's shared memory is used for."""
    assert eb.balance_workspace_size(T, E, 1 if off is None else len(off) - 1) > 0
    _check(cuda_dev, *_inputs(T, E, k, seed=T + E), off=off)


def test_more_tokens_than_one_wave(cuda_dev):
    """Past 64 rows for each of the card's teams: more CTAs than SMs, against sums in binary64 on the GPU."""
    T, E, k = 160000, 16, 2
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    x = torch.randn(T, E, generator=g, device=cuda_dev)
    mask = (torch.rand(T, generator=g, device=cuda_dev) > 0.1).to(torch.uint8)
    ids = torch.topk(x, k, dim=1).indices.to(torch.int32)
    loss, counts, probs, n = eb.moe_balance_loss(x, ids, mask, 0.1)
    s = torch.sigmoid(x.double())
    p = s / s.sum(1, keepdim=True) * mask.double()[:, None]
    want = p.sum(0)
    assert int(n) == int(mask.sum())
    assert torch.equal(counts[0].long(), torch.bincount(ids[mask != 0].flatten().long(), minlength=E))
    tol = (float(x.abs().max()) + 40 + 72 + T / 128 + 16) * U
    assert bool(((probs[0].double() - want).abs() <= tol * want).all())
    wl = 0.1 * E / (k * float(n) ** 2) * float((counts[0].double() * want).sum())
    assert abs(float(loss) - wl) <= (tol + 20 * U) * wl
    dw = torch.randn(T, k, generator=g, device=cuda_dev)
    got = eb.moe_route_backward(x, ids, mask, grad_weights=dw)
    sj = torch.gather(s, 1, ids.long())
    w = sj / sj.sum(1, keepdim=True)
    part = w * (1 - sj) * (dw.double() - (dw.double() * w).sum(1, keepdim=True)) * mask.double()[:, None]
    ref = torch.zeros_like(s).scatter_add_(1, ids.long(), part)
    assert float((got.double() - ref).norm() / ref.norm()) < 60 * U


@pytest.mark.parametrize("T,E", [(4096, 8), (4097, 8), (9000, 8), (2000, 128), (2049, 128), (1024, 256), (1025, 256)])
def test_around_the_cluster_sizes(cuda_dev, T, E):
    """The largest batches of one cluster and the next larger ones count every token."""
    _check(cuda_dev, *_inputs(T, E, 2, seed=T), off=[0, T // 3, T])


def test_every_token_masked(cuda_dev):
    x, ids, mask, dw = _inputs(20, 40, 4, seed=1)
    mask[:] = 0
    x[:] = np.nan
    _check(cuda_dev, x, ids, mask, dw, off=[0, 5, 20])


@pytest.mark.parametrize("shift", [-40.0, -60.0, -85.0, -300.0, 60.0, 300.0])
@pytest.mark.parametrize("E", [64, 1000])
def test_saturated_logits(cuda_dev, shift, E):
    """All sigmoids next to 0 (their ratios stay) or to 1 (no gradient is left)."""
    _check(cuda_dev, *_inputs(30, E, 4, seed=7, shift=shift))


def test_infinite_logits(cuda_dev):
    x, ids, mask, dw = _inputs(24, 40, 4, seed=5, masked=0.0)
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, 3:9] = np.inf
    x[3] = np.inf
    x[4, ::2] = -np.inf
    _check(cuda_dev, x, ids, mask, dw)


def test_odd_picks(cuda_dev):
    """Repeated ids, ids outside [0, E), rows without a pick."""
    x, ids, mask, dw = _inputs(50, 40, 6, seed=9)
    ids[3] = 5
    ids[4, :3] = 7
    ids[5] = -1
    ids[6, 2:] = 40
    ids[7, 0] = 2 ** 31 - 1
    ids[8] = -2 ** 31
    ids[9, ::2] = ids[9, 1]
    _check(cuda_dev, x, ids, mask, dw)


def test_gradient_along_a_direction(cuda_dev):
    """The GPU's gradient against the difference quotient of the loss in binary64."""
    x, ids, mask, _ = _inputs(60, 24, 3, seed=2, masked=0.1)
    off = [0, 20, 60]
    x = np.where(mask[:, None] != 0, x, 0).astype(np.float32)
    tx, ti, tm, to = _dev(cuda_dev, x, ids, mask, np.asarray(off, np.int32))
    _, counts, _, n = eb.moe_balance_loss(tx, ti, tm, 1.0, seq_offsets=to)
    g = eb.moe_route_backward(tx, ti, tm, grad_loss=torch.ones(1, device=cuda_dev), coeff=1.0, counts=counts,
                              seq_tokens=n, seq_offsets=to).cpu().numpy().astype(np.float64)
    d = np.random.default_rng(4).normal(size=x.shape)
    h = 1e-4
    num = (balance(x + h * d, ids, mask, 1.0, off)[0] - balance(x - h * d, ids, mask, 1.0, off)[0]) / (2 * h)
    assert abs((g * d).sum() - num) <= 1e-5 * np.abs(g * d).sum()


def test_repeats_bit_for_bit_and_leaves_guards(cuda_dev):
    """The same bits on every run, on a side stream, and replayed from a graph; nothing behind the outputs changes."""
    T, E, k, off = 3000, 260, 8, [0, 700, 701, 2900]
    x, ids, mask, dw = _inputs(T, E, k, seed=11)
    tx, ti, tm, tw, to = _dev(cuda_dev, x, ids, mask, dw, np.asarray(off, np.int32))
    Q = len(off) - 1
    sizes = {"loss": 1, "counts": Q * E, "prob_sums": Q * E, "seq_tokens": Q, "grad": T * E}
    buf = {n: torch.full((s + 64,), -77, dtype=torch.int32 if n in ("counts", "seq_tokens") else torch.float32,
                         device=cuda_dev) for n, s in sizes.items()}
    out = {n: buf[n][:s] for n, s in sizes.items()}
    out["counts"], out["prob_sums"] = out["counts"].view(Q, E), out["prob_sums"].view(Q, E)
    out["grad"] = out["grad"].view(T, E)
    need = eb.balance_workspace_size(T, E, Q)
    assert need > 0
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device=cuda_dev)
    one = torch.ones(1, device=cuda_dev)

    def step():
        eb.moe_balance_loss(tx, ti, tm, 0.1, seq_offsets=to, loss=out["loss"], counts=out["counts"],
                            prob_sums=out["prob_sums"], seq_tokens=out["seq_tokens"], workspace=ws[:need])
        eb.moe_route_backward(tx, ti, tm, grad_weights=tw, grad_loss=one, coeff=0.1, counts=out["counts"],
                              seq_tokens=out["seq_tokens"], seq_offsets=to, grad_logits=out["grad"])
    step()
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in out.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(out[n], first[n]) for n in out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in out.values():
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], first[n]) for n in out)
    assert all(bool((buf[n][s:] == -77).all()) for n, s in sizes.items()) and bool((ws[need:] == 77).all())


@pytest.mark.parametrize("T,E", [(40, 64), (3000, 128), (60, 2560)])
def test_addresses_of_16_bytes(cuda_dev, T, E):
    """Inputs and outputs at addresses that are 16-byte aligned and no more give the same bits."""
    x, ids, mask, dw = _inputs(T, E, 4, seed=8)
    tx, ti, tm, tw = _dev(cuda_dev, x, ids, mask, dw)

    def shifted(t):
        buf = torch.zeros(t.numel() + 64, dtype=t.dtype, device=cuda_dev)
        step = 16 // t.element_size()
        at = next(k for k in range(step, 64, step) if (buf.data_ptr() + k * t.element_size()) % 32 == 16)
        buf[at:at + t.numel()].copy_(t.flatten())
        return buf[at:at + t.numel()].view(t.shape)
    one = torch.ones(1, device=cuda_dev)
    out = []
    for f in (lambda t: t, shifted):
        b = tuple(f(t) for t in (tx, ti, tm))
        loss, counts, probs, n = eb.moe_balance_loss(*b, 0.1)
        out.append((loss, counts, probs, n, eb.moe_route_backward(*b, grad_weights=f(tw), grad_loss=one, coeff=0.1,
                                                                  counts=f(counts), seq_tokens=f(n),
                                                                  grad_logits=f(torch.zeros(T, E, device=cuda_dev)))))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*out))


def test_two_streams_at_once(cuda_dev):
    """Calls that overlap on the GPU, one cluster and many CTAs."""
    cases = [_dev(cuda_dev, *_inputs(T, E, 6, seed=T)) for T, E in ((100, 64), (4000, 256), (200, 512), (300, 2560))]
    one = torch.ones(1, device=cuda_dev)

    def step(x, ids, mask, dw):
        loss, counts, probs, n = eb.moe_balance_loss(x, ids, mask, 0.1)
        return loss, counts, probs, n, eb.moe_route_backward(x, ids, mask, grad_weights=dw, grad_loss=one, coeff=0.1,
                                                             counts=counts, seq_tokens=n)
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for s, c, g in zip(streams, cases, got):
            with torch.cuda.stream(s):
                g.append(step(*c))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for w, g in zip(want, got) for r in g for p, q in zip(w, r))
    assert eb.device_status() == 0


def test_no_tokens(cuda_dev):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=cuda_dev)  # noqa: E731
    off = z(3, dt=torch.int32)
    loss, counts, probs, n = eb.moe_balance_loss(z(0, 16), z(0, 2, dt=torch.int32), z(0, dt=torch.uint8), 0.1,
                                                 seq_offsets=off)
    torch.cuda.synchronize()
    assert float(loss) == 0 and not counts.any() and not probs.any() and not n.any()
    g = eb.moe_route_backward(z(0, 16), z(0, 2, dt=torch.int32), z(0, dt=torch.uint8), grad_weights=z(0, 2))
    assert g.shape == (0, 16)


def test_broken_offsets_stay_in_bounds(cuda_dev):
    """Offsets that are not ascending or lie outside the batch: any values, but no access out of range."""
    x, ids, mask, dw = _inputs(64, 32, 4, seed=1)
    tx, ti, tm, to = _dev(cuda_dev, x, ids, mask, np.asarray([50, -9, 400, 3, 2 ** 31 - 1, 10], np.int32))
    _, counts, _, n = eb.moe_balance_loss(tx, ti, tm, 0.1, seq_offsets=to)
    eb.moe_route_backward(tx, ti, tm, grad_loss=torch.ones(1, device=cuda_dev), coeff=0.1, counts=counts,
                          seq_tokens=n, seq_offsets=to)
    torch.cuda.synchronize()
    assert eb.device_status() == 0


def test_the_gate_and_its_training_together(cuda_dev):
    """moe_route, the balance loss of its picks and the gradient that reaches the logits, in one go."""
    T, E, k = 500, 256, 8
    r = np.random.default_rng(0)
    x = r.normal(size=(T, E)).astype(np.float32)
    mask = (r.random(T) > 0.1).astype(np.uint8)
    tx, tm, bias, dw = _dev(cuda_dev, x, mask, (0.1 * r.random(E)).astype(np.float32),
                            r.normal(size=(T, k)).astype(np.float32))
    ids, w = eb.moe_route(tx, bias, tm, k)
    loss, counts, _, n = eb.moe_balance_loss(tx, ids, tm, 0.01)
    grad = eb.moe_route_backward(tx, ids, tm, grad_weights=dw, grad_loss=torch.ones(1, device=cuda_dev), coeff=0.01,
                                 counts=counts, seq_tokens=n)
    offsets, _, _ = eb.moe_dispatch(ids, E)
    torch.cuda.synchronize()
    assert torch.equal(counts[0], offsets[1:] - offsets[:-1])     # the dispatch counts the same picks
    rg, mag = backward(x, ids.cpu().numpy(), mask, dw.cpu().numpy(), 1.0, 0.01, counts.cpu().numpy(), n.cpu().numpy())
    assert np.all(np.abs(grad.cpu().numpy() - rg) <= (2 * (_xmax(x) + 40) + 60) * U * mag + 1e-37)
    # the weights that the gradient is taken of are the gate's
    sj = 1 / (1 + np.exp(-np.take_along_axis(x.astype(np.float64), np.maximum(ids.cpu().numpy(), 0), 1)))
    assert np.allclose(w.cpu().numpy()[mask != 0], (sj / sj.sum(1, keepdims=True))[mask != 0], rtol=1e-6)


@pytest.mark.parametrize("grad_loss", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,E,k", [(60, 40, 4), (60, 37, 4), (70, 512, 22), (60, 2560, 8)])
def test_overflowed_loss_gradient_stays_in_its_sequences(cuda_dev, grad_loss, T, E, k):
    """Rows of invalid tokens stay zero and rows of no sequence keep the gate's part alone."""
    x, ids, mask, dw = _inputs(T, E, k, seed=6)
    off = [7, 30, 30, 45]
    tx, ti, tm, tw, to = _dev(cuda_dev, x, ids, mask, dw, np.asarray(off, np.int32))
    _, counts, _, n = eb.moe_balance_loss(tx, ti, tm, 0.1, seq_offsets=to)
    gl = torch.tensor([grad_loss], device=cuda_dev)
    rest = dict(grad_loss=gl, coeff=0.1, counts=counts, seq_tokens=n, seq_offsets=to)
    both = eb.moe_route_backward(tx, ti, tm, grad_weights=tw, **rest)
    bal = eb.moe_route_backward(tx, ti, tm, **rest)
    gate = eb.moe_route_backward(tx, ti, tm, grad_weights=tw)
    torch.cuda.synchronize()
    t = torch.arange(T, device=cuda_dev)
    inside = (tm != 0) & (t >= off[0]) & (t < off[-1])
    assert not both[tm == 0].any() and not bal[~inside].any()
    assert torch.equal(both[~inside], gate[~inside])
    # counts of 0 beside others: inf * 0 in the row's mean, so the formula is NaN all over the row
    assert bool((counts == 0).any(1)[n > 0].all())
    assert bool(both[inside].isnan().all()) and bool(bal[inside].isnan().all())


@pytest.mark.parametrize("T,E", [(30, 8), (30, 37), (30, 600), (4000, 256), (300, 2560), (200, 3001)])
@pytest.mark.parametrize("kind", ["all", "beside -inf", "beside numbers"])
def test_nan_logits_of_a_valid_token_reach_the_loss(cuda_dev, T, E, kind):
    """A row of NaN is no row of -inf: its sequence's sums and the loss are NaN, another sequence's sums are not."""
    x, ids, mask, dw = _inputs(T, E, 4, seed=3)
    mask[[2, T - 1]] = 1
    x[2], x[T - 1] = np.nan, 0.0
    if kind == "beside -inf":
        x[2, 1:] = -np.inf
    if kind == "beside numbers":
        x[2, 1:] = np.linspace(-3, 3, E - 1)
    off = [0, T // 2, T]
    tx, ti, tm, tw, to = _dev(cuda_dev, x, ids, mask, dw, np.asarray(off, np.int32))
    loss, counts, probs, n = eb.moe_balance_loss(tx, ti, tm, 0.1, seq_offsets=to)
    g = eb.moe_route_backward(tx, ti, tm, grad_loss=torch.ones(1, device=cuda_dev), coeff=0.1, counts=counts,
                              seq_tokens=n, seq_offsets=to)
    torch.cuda.synchronize()
    assert bool(loss.isnan().all()) and bool(probs[0].isnan().all()) and bool(probs[1].isfinite().all())
    rows = torch.arange(T, device=cuda_dev) != 2
    assert bool(g[2].isnan().all()) and bool(g[rows].isfinite().all())


def test_loss_gradient_without_its_coefficient_is_refused(cuda_dev):
    """Not a silent gradient of zero: grad_loss comes with the loss call's coeff, counts and seq_tokens."""
    x, ids, mask, dw = _inputs(20, 16, 2, seed=1)
    tx, ti, tm, tw = _dev(cuda_dev, x, ids, mask, dw)
    _, counts, _, n = eb.moe_balance_loss(tx, ti, tm, 0.1)
    good = dict(grad_loss=torch.ones(1, device=cuda_dev), coeff=0.1, counts=counts, seq_tokens=n)
    assert eb.moe_route_backward(tx, ti, tm, **good).any()
    for name in ("coeff", "counts", "seq_tokens"):
        with pytest.raises(ValueError, match="grad_loss needs"):
            eb.moe_route_backward(tx, ti, tm, **{k: v for k, v in good.items() if k != name})
    eb.moe_route_backward(tx, ti, tm, grad_weights=tw)         # the gate alone needs none


def test_inside_an_autograd_function(cuda_dev):
    """The loss and its gradient as one node of a caller's graph: the parameters below it get the formula's gradient."""
    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids, mask):
            loss, counts, _, n = eb.moe_balance_loss(logits, ids, mask, 0.5)
            ctx.save_for_backward(logits, ids, mask, counts, n)
            return loss

        @staticmethod
        def backward(ctx, g):
            logits, ids, mask, counts, n = ctx.saved_tensors
            return eb.moe_route_backward(logits, ids, mask, grad_loss=g, coeff=0.5, counts=counts, seq_tokens=n), None, None

    x, ids, mask, _ = _inputs(40, 24, 3, seed=2, masked=0.1)
    x = np.where(mask[:, None] != 0, x, 0).astype(np.float32)
    tx, ti, tm = _dev(cuda_dev, x, ids, mask)
    tx.requires_grad_()
    with pytest.raises(ValueError, match="require a gradient"):
        eb.moe_balance_loss(tx, ti, tm, 0.5)
    (3.0 * Balance.apply(tx, ti, tm)).sum().backward()
    _, counts, _, n = balance(x, ids, mask, 0.5)
    want, mag = backward(x, ids, mask, grad_loss=3.0, coeff=0.5, counts=counts, seq_tokens=n)
    assert np.all(np.abs(tx.grad.cpu().numpy() - want) <= (2 * (_xmax(x) + 40) + 60) * U * mag + 1e-37)
