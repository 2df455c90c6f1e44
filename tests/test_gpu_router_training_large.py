"""Balance loss and gate gradient where a team of warps takes many rows: its
ring of copied rows, its ring of lists and its two join buffers wrap, in one
wave of CTAs and in several, against binary64 formed on the GPU.

Tolerances in units u = 2^-24: a probability is off by at most (max|x| + 40) u
(as for the small batches).  Of positive FP32 terms, a team adds at most 128
rows in a register, then come at most 24 teams, the slots of a sequence (one
per CTA) in 16 runs, and the 16 runs: 128 + 24 + CTAs / 16 + 16 roundings.  The
loss adds 5 + E / 32 + Q + 8.  A gradient: two terms of each g - G, the slope
and the gate's part, (2 (max|x| + 40) + 60) u of the sum of magnitudes.
"""
import pytest
import torch

import expert_combine_b200 as eb

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SMS, ROWS = 148, 128          # CTAs of a wave, most rows that a team adds up in one


def _rows_per_team(T, E, warps):
    """-> (rows a team, CTAs) with teams of ceil(E / 512) warps."""
    teams = warps // -(-E // 512)
    waves = -(-T // (SMS * teams * ROWS))
    rows = -(-T // (SMS * teams * waves))
    return rows, -(-T // (rows * teams))


def _inputs(dev, T, E, k, Q, far):
    g = torch.Generator(device=dev).manual_seed(T + E)
    x = 2.0 * torch.randn(T, E, generator=g, device=dev)
    if far:                                               # rows that are done over, between others
        x[::5] -= 60.0
        x[::13, E // 2:] = -float("inf")
    mask = (torch.rand(T, generator=g, device=dev) >= 0.1).to(torch.uint8)
    ids = torch.topk(x, k, dim=1).indices.to(torch.int32)
    ids[::7, 0] = -1
    if k > 1:
        ids[3::11, 1] = ids[3::11, 0]                     # an expert picked twice
    x[mask == 0] = float("nan")                           # never used
    cuts = torch.sort(torch.randint(0, T + 1, (Q + 1,), generator=g, device=dev)).values
    cuts[1] = cuts[2]                                     # one empty sequence; tokens before the first and behind the last
    return x, ids, mask, torch.randn(T, k, generator=g, device=dev), cuts.to(torch.int32)


def _check(dev, T, E, k, Q, far=False):
    x, ids, mask, dw, cuts = _inputs(dev, T, E, k, Q, far)
    coeff, gl = 0.3, 1.25
    loss, counts, probs, n = eb.moe_balance_loss(x, ids, mask, coeff, seq_offsets=cuts)
    got = eb.moe_route_backward(x, ids, mask, grad_weights=dw, grad_loss=torch.tensor([gl], device=dev), coeff=coeff,
                                counts=counts, seq_tokens=n, seq_offsets=cuts)
    torch.cuda.synchronize()
    f = torch.float64
    seq = torch.searchsorted(cuts, torch.arange(T, device=dev, dtype=torch.int32), right=True) - 1
    live = (mask != 0) & (seq >= 0) & (seq < Q)
    xmax = float(x[x.isfinite()].abs().max())
    ok = (ids >= 0) & (ids < E)
    # counts and valid tokens
    q_of = torch.where(live, seq, Q)
    hist = torch.zeros((Q + 1) * E + 1, dtype=torch.int64, device=dev)
    flat = torch.where(ok, q_of[:, None] * E + ids, (Q + 1) * E)
    hist.scatter_add_(0, flat.flatten(), torch.ones_like(flat).flatten())
    assert torch.equal(counts.long().flatten(), hist[:Q * E])
    assert torch.equal(n.long(), torch.bincount(q_of, minlength=Q + 1)[:Q])
    # g of every sequence; none outside
    some = max(1, int((n > 0).sum()))
    per = torch.where(n > 0, gl * coeff / some * E / (k * n.to(f).clamp(min=1) ** 2), 0.0)
    g = torch.cat([counts.to(f) * per[:, None], torch.zeros(1, E, dtype=f, device=dev)])
    want_p = torch.zeros(Q + 1, E, dtype=f, device=dev)
    each = xmax + 40
    for t0 in range(0, T, 8192):
        t = slice(t0, t0 + 8192)
        s = torch.sigmoid(torch.where(mask[t, None] != 0, x[t], 0.0).to(f))
        S = s.sum(1, keepdim=True)
        p = s / S
        want_p.index_add_(0, q_of[t], p)
        gt = g[q_of[t]]
        G = (gt * p).sum(1, keepdim=True)
        grad, mag = (gt - G) * p * (1 - s), (gt + G) * p * (1 - s)
        pick = mask[t, None].bool() & ok[t]
        at = ids[t].long().clamp(min=0)
        sj = s.gather(1, at) * pick
        w = sj / sj.sum(1, keepdim=True).clamp(min=1e-300)
        d = torch.where(pick, dw[t], 0.0).to(f)
        om = 1 - s.gather(1, at)
        grad.scatter_add_(1, at, w * om * (d - (d * w).sum(1, keepdim=True)))
        mag.scatter_add_(1, at, w * om * (d.abs() + (d.abs() * w).sum(1, keepdim=True)))
        grad[mask[t] == 0], mag[mask[t] == 0] = 0.0, 0.0
        assert bool(((got[t].to(f) - grad).abs() <= (2 * each + 60) * U * mag + 1e-37).all()), t0
    tol = (each + 128 + 24 + _rows_per_team(T, E, 24)[1] / 16 + 16) * U
    assert bool(((probs.to(f) - want_p[:Q]).abs() <= tol * want_p[:Q] + 1e-37).all())
    nn = n.to(f)
    wl = coeff / some * float((torch.where(nn > 0, E / (k * nn.clamp(min=1) ** 2), 0.0) *
                               (counts.to(f) * want_p[:Q]).sum(1)).sum())
    assert abs(float(loss) - wl) <= (tol + (5 + E / 32 + Q + 8) * U) * wl
    assert eb.device_status() == 0


@pytest.mark.parametrize("T,E,k", [(12000, 2560, 8), (9000, 4096, 32), (11000, 3001, 8), (40000, 512, 22),
                                   (40000, 511, 4), (30000, 1000, 5)])
def test_many_rows_a_team(cuda_dev, T, E, k):
    lists = 4 * (4 if k <= 8 else 2 if k <= 16 else 1)    # rows that a team's ring of lists holds; its ring of rows: 8
    assert _rows_per_team(T, E, 24)[0] > 8 and _rows_per_team(T, E, 16)[0] > max(8, lists)
    assert _rows_per_team(T, E, 24)[1] <= SMS and _rows_per_team(T, E, 16)[1] <= SMS
    _check(cuda_dev, T, E, k, Q=6)


@pytest.mark.parametrize("T,E,k", [(500000, 16, 2), (500001, 17, 3), (80000, 2560, 8)])
def test_several_waves(cuda_dev, T, E, k):
    for warps in (24, 16):
        assert _rows_per_team(T, E, warps)[1] > SMS
    one = (SMS + 6) * E * 8                               # bytes of the sums of one wave's slots
    assert eb.balance_workspace_size(T, E, 6) > one * 1.5
    _check(cuda_dev, T, E, k, Q=6)


@pytest.mark.parametrize("T,E,k", [(12000, 2560, 8), (11000, 3001, 8), (40000, 512, 22), (40000, 66, 6)])
def test_rows_far_below_zero_between_others(cuda_dev, T, E, k):
    _check(cuda_dev, T, E, k, Q=6, far=True)
