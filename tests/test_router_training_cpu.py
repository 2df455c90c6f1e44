"""Balance loss and gate gradient without a GPU: the binary64 formulas against
differences, and the refusals of the library and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import expert_combine_b200 as eb
from router_training import backward, balance

F32, I32, U8 = torch.float32, torch.int32, torch.uint8


def _case(T=11, E=13, k=3, seed=0):
    r = np.random.default_rng(seed)
    x = r.normal(size=(T, E)) * 2
    ids = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    mask = np.ones(T, bool)
    mask[[2, 7]] = False
    return x, ids, mask, r


def test_loss_gradient_is_the_difference_quotient():
    x, ids, mask, r = _case()
    off = [1, 4, 4, 9]                         # tokens 0, 9, 10 belong to no sequence; one sequence is empty
    loss, counts, _, n = balance(x, ids, mask, 0.3, off)
    grad, _ = backward(x, ids, mask, grad_loss=1.7, coeff=0.3, counts=counts, seq_tokens=n, offsets=off)
    for _ in range(5):
        d = r.normal(size=x.shape)
        h = 1e-5
        num = (balance(x + h * d, ids, mask, 0.3, off)[0] - balance(x - h * d, ids, mask, 0.3, off)[0]) / (2 * h)
        assert abs(1.7 * num - (grad * d).sum()) < 1e-7 * (1 + abs(num))
    assert not grad[[0, 2, 7, 9, 10]].any()


def test_gate_gradient_is_the_difference_quotient():
    x, ids, mask, r = _case()
    ids[3, 1] = ids[3, 0]                      # an expert picked twice
    ids[4, 2] = -1
    dw = r.normal(size=ids.shape)
    grad, _ = backward(x, ids, mask, grad_w=dw)

    def value(x):
        total = 0.0
        for t in range(len(x)):
            ok = ids[t] >= 0
            if mask[t]:
                s = 1 / (1 + np.exp(-x[t, ids[t][ok]]))
                total += (dw[t][ok] * s / s.sum()).sum()
        return total
    for _ in range(5):
        d = r.normal(size=x.shape)
        h = 1e-5
        assert abs((value(x + h * d) - value(x - h * d)) / (2 * h) - (grad * d).sum()) < 1e-7


def test_host_tensors_and_wrong_types_are_refused():
    T, E, k = 4, 16, 2
    good = (torch.zeros(T, E), torch.zeros(T, k, dtype=I32), torch.ones(T, dtype=U8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        eb.moe_balance_loss(*good, 0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        eb.moe_route_backward(*good, grad_weights=torch.zeros(T, k))
    with pytest.raises(TypeError, match="expected"):
        eb.moe_balance_loss(good[0].to(torch.bfloat16), *good[1:], 0.1)
    with pytest.raises(TypeError, match="expected"):
        eb.moe_route_backward(good[0].to(torch.float64), *good[1:])


def test_library_refuses_before_any_launch():
    lib = eb.load()
    N, a, odd = None, ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)
    Z, big = ctypes.c_size_t(0), ctypes.c_size_t(1 << 40)

    def loss(T=4, E=16, k=2, off=N, Q=1, ptr=a, out=a, ws=a, size=big):
        return lib.moe_balance_loss(ptr, ptr, ptr, T, E, k, off, Q, 0.1, out, out, out, out, ws, size, N)
    assert loss(T=-1) == 1 and loss(Q=-1) == 1
    assert loss(E=1) == 2 and loss(E=4097) == 2 and loss(k=33, E=64) == 2 and loss(k=0) == 2 and loss(Q=0) == 2
    assert loss(T=1 << 29, k=8) == 2 and loss(Q=1 << 20, E=4096, off=a) == 2
    assert loss(Q=3) == 1 and "seq_offsets" in eb.last_error()
    assert loss(ptr=N) == 1 and "null" in eb.last_error()
    assert loss(out=N) == 1 and loss(out=odd) == 1 and loss(ptr=odd) == 1 and loss(off=odd, Q=2) == 1
    T = 100000                                                  # a batch that needs a workspace
    assert loss(T=T, ws=N) == 1 and "workspace" in eb.last_error()
    need = eb.balance_workspace_size(T, 16, 1)
    assert need > 0 and loss(T=T, size=ctypes.c_size_t(need - 1)) == 1 and loss(T=T, size=Z) == 1
    assert loss(T=T, ws=odd) == 1 and "aligned" in eb.last_error()
    assert eb.balance_workspace_size(4, 16, 1) == 0
    assert eb.balance_workspace_size(4, 5000, 1) == 0 and eb.balance_workspace_size(4, 16, 0) == 0

    b = ctypes.c_void_p(1 << 32)

    def back(T=4, E=16, k=2, ptr=a, dw=a, dl=a, counts=a, n=a, off=N, Q=1, out=b):
        return lib.moe_route_backward(ptr, ptr, ptr, T, E, k, dw, dl, 0.1, counts, n, off, Q, out, N)
    assert back(T=0) == 0                                       # empty: no launch
    assert back(dw=N, dl=N) == 1 and "neither" in eb.last_error()
    assert back(counts=N) == 1 and back(n=N) == 1 and back(out=N) == 1 and back(ptr=N) == 1
    for p in (a, ctypes.c_void_p(0x1000 + 16), ctypes.c_void_p(0x1000 - 16)):
        assert back(out=p) == 1 and "overlaps" in eb.last_error()
    assert back(Q=2) == 1 and back(E=4097) == 2 and back(T=-1) == 1 and back(k=17) == 2
    assert back(ptr=odd) == 1 and back(dw=odd) == 1 and back(out=odd) == 1
    assert eb.supported(eb.STAGE_BALANCE, 8192, 0, 256, 8, 4) and not eb.supported(eb.STAGE_BALANCE, 1, 0, 4, 8, 1)


def test_gradient_over_any_input_is_refused():
    """grad_logits may share no byte with what other CTAs still read."""
    lib = eb.load()
    T, E, k, Q = 4, 16, 2, 3
    at = {n: (i + 1) << 32 for i, n in enumerate(("x", "ids", "mask", "dw", "dl", "counts", "n", "off"))}
    size = {"x": T * E * 4, "ids": T * k * 4, "mask": T, "dw": T * k * 4, "dl": 4, "counts": Q * E * 4, "n": Q * 4,
            "off": (Q + 1) * 4}
    P = {n: ctypes.c_void_p(a) for n, a in at.items()}

    def back(out):
        return lib.moe_route_backward(P["x"], P["ids"], P["mask"], T, E, k, P["dw"], P["dl"], 0.1, P["counts"], P["n"],
                                      P["off"], Q, ctypes.c_void_p(out), None)
    for n in at:
        last = (at[n] + size[n] - 1) & ~15
        for out in (at[n], last, at[n] - T * E * 4 + 16):
            assert back(out) == 1 and "overlaps" in eb.last_error(), n


def test_loss_outputs_over_another_array_are_refused():
    """Outputs and workspace may share no byte with an input or with one another."""
    lib = eb.load()
    T, E, k, Q = 100000, 16, 2, 3
    need = eb.balance_workspace_size(T, E, Q)
    assert need > 0
    size = {"x": T * E * 4, "ids": T * k * 4, "mask": T, "off": (Q + 1) * 4, "loss": 4, "counts": Q * E * 4,
            "probs": Q * E * 4, "n": Q * 4, "ws": need}
    at = {n: (i + 1) << 32 for i, n in enumerate(size)}

    def loss(**moved):
        p = {n: ctypes.c_void_p(a) for n, a in {**at, **moved}.items()}
        return lib.moe_balance_loss(p["x"], p["ids"], p["mask"], T, E, k, p["off"], Q, 0.1, p["loss"], p["counts"],
                                    p["probs"], p["n"], p["ws"], ctypes.c_size_t(need), None)
    for out in ("loss", "counts", "probs", "n", "ws"):
        for other in size:
            if other != out:
                for where in (at[other], (at[other] + size[other] - 1) & ~15, at[other] - ((size[out] - 1) & ~15)):
                    assert loss(**{out: where}) == 1 and "overlaps" in eb.last_error(), (out, other)


def test_a_loss_that_would_lose_its_gradient_is_refused():
    """logits that require a gradient, while gradients are recorded; detached or without recording they go on."""
    T, E, k = 4, 16, 2
    x = torch.zeros(T, E, requires_grad=True)
    rest = (torch.zeros(T, k, dtype=I32), torch.ones(T, dtype=U8), 0.1)
    for logits in (x, x * 2):
        with pytest.raises(ValueError, match="moe_route_backward"):
            eb.moe_balance_loss(logits, *rest)
    with pytest.raises(ValueError, match="CUDA tensor"):
        eb.moe_balance_loss(x.detach(), *rest)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        eb.moe_balance_loss(x, *rest)
