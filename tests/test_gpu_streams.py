"""Calls with a `stream` argument other than the current stream: what they
allocate belongs to that stream, also the workspace that they drop on return."""
import pytest
import torch

import expert_combine_b200 as eb

pytestmark = pytest.mark.gpu


def _calls(dev):
    """name -> call(**kw) that allocates its outputs and, for the first three, a workspace."""
    g = torch.Generator(device=dev).manual_seed(3)
    T, E, k, H, R, L = 3000, 256, 8, 512, 16, 6
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    logits, x = rnd(T, E), rnd(T, H).to(torch.bfloat16)
    mask = torch.ones(T, dtype=torch.uint8, device=dev)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    a, b = rnd(L, R, H).to(torch.bfloat16), rnd(L, E, R).to(torch.bfloat16)
    of = torch.randint(-1, L, (T,), generator=g, device=dev, dtype=torch.int32)
    w3 = eb.router_weight_prepare(rnd(E, H))
    bias, dw = rnd(E), rnd(T, k)
    return {"lora_add": lambda **kw: eb.lora_add(logits, x, a, b, of, **kw),
            "moe_balance_loss": lambda **kw: eb.moe_balance_loss(logits, ids, mask, 0.1, **kw),
            "moe_dispatch": lambda **kw: eb.moe_dispatch(ids, E, **kw),
            "moe_route": lambda **kw: eb.moe_route(logits, bias, mask, k, **kw),
            "moe_route_backward": lambda **kw: eb.moe_route_backward(logits, ids, mask, grad_weights=dw, **kw),
            "router_logits": lambda **kw: eb.router_logits(x, w3, **kw)}


NAMES = ("lora_add", "moe_balance_loss", "moe_dispatch", "moe_route", "moe_route_backward", "router_logits")


def _flat(result):
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_made_on_the_call_s_stream(cuda_dev, monkeypatch, name):
    call = _calls(cuda_dev)[name]
    want = _flat(call())
    seen = []
    for maker in ("empty", "empty_like"):
        plain = getattr(torch, maker)
        monkeypatch.setattr(torch, maker, lambda *a, _f=plain, **kw: (seen.append(torch.cuda.current_stream()),
                                                                      _f(*a, **kw))[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _flat(call(stream=side))
    inside, seen[:] = list(seen), []
    assert torch.cuda.current_stream() != side
    torch.cuda.synchronize()
    call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert inside and all(s == side for s in inside)
    assert len(seen) == len(inside) and all(s != side for s in seen)
    assert all(torch.equal(w, o) for w, o in zip(want, got))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_s_later_memory_is_other_memory(cuda_dev, name):
    """Tensors allocated and overwritten right after the call, while it is still to run, do not change its result."""
    call = _calls(cuda_dev)[name]
    want = _flat(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)            # about a millisecond
        got = _flat(call(stream=side))
        sizes = [eb.lora_workspace_size(3000, 512, 256, 16, 6), eb.balance_workspace_size(3000, 256, 1),
                 eb.dispatch_workspace_size(3000, 8, 256)]
        for n in sizes * 4:
            torch.empty(n, dtype=torch.uint8, device=cuda_dev).fill_(255)
        side.synchronize()
        assert all(torch.equal(w, o) for w, o in zip(want, got))
    torch.cuda.synchronize()
    assert eb.device_status() == 0


def test_stream_as_a_positional_argument(cuda_dev):
    call = _calls(cuda_dev)["router_logits"]
    want = call()
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    x = torch.randn(16, 64, generator=g, device=cuda_dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=torch.cuda.ExternalStream(side.cuda_stream))
    w3 = eb.router_weight_prepare(x, None, side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(w3, eb.router_weight_prepare(x))


def test_the_current_stream_and_device_come_back(cuda_dev):
    """Also after a refused call; outputs that the caller gave are the ones returned."""
    x = torch.randn(16, 64, device=cuda_dev)
    w3 = torch.empty(3, 16, 64, dtype=torch.bfloat16, device=cuda_dev)
    before, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(before):
        assert eb.router_weight_prepare(x, w3, stream=side) is w3
        assert torch.cuda.current_stream() == before and torch.cuda.current_device() == cuda_dev.index
        with pytest.raises(ValueError, match="contiguous"):
            eb.router_weight_prepare(x.t(), stream=side)
        assert torch.cuda.current_stream() == before and torch.cuda.current_device() == cuda_dev.index
    torch.cuda.synchronize()
