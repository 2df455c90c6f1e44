"""lora_add on the GPU against its definition in binary64.

Tolerance, with u = 2^-24 (half a step of binary32): a product of BF16 values
is exact; a tensor-core accumulation is off by at most one step (2 u) of the
terms summed so far each 16 products, so v is off by (H / 16 + 16) 2 u times
sum_h |x A| (partial sums joined in FP32 are among the 16).  The second product
adds R / 8 + 8 steps, the scale and the parts v may be split into another 2^-23
(2^-15 for BF16 outputs), all times sum_r |v B|.  The result is rounded once:
u |out|, or 2^-8 |out| for BF16.
"""
import pytest
import torch

import expert_combine_b200 as eb

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(dev, T, H, N, R, L, bf16, seed=0, ids=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if ids is None:
        ids = torch.randint(-1, L, (T,), generator=g, device=dev)
    return dict(base=rnd(T, N).to(torch.bfloat16 if bf16 else torch.float32), x=rnd(T, H).to(torch.bfloat16),
                a=(rnd(L, R, H) * H ** -0.5).to(torch.bfloat16), b=(rnd(L, N, R) * R ** -0.5).to(torch.bfloat16),
                adapter_ids=torch.as_tensor(ids, dtype=torch.int32).to(dev),
                scales=0.25 + torch.rand(L, generator=g, device=dev))


def _reference(i):
    """-> (out in binary64, its tolerance)."""
    f = torch.float64
    T, H = i["x"].shape
    L, R = i["a"].shape[:2]
    bf16 = i["base"].dtype == torch.bfloat16
    out, tol = i["base"].to(f).clone(), torch.zeros_like(i["base"], dtype=f)
    for a in range(L):
        t = torch.nonzero(i["adapter_ids"] == a).flatten()
        if len(t) == 0:
            continue
        s = 1.0 if i["scales"] is None else float(i["scales"][a].to(f))
        x, A, B = i["x"][t].to(f), i["a"][a].to(f), i["b"][a].to(f)
        v = x @ A.T
        out[t] += s * (v @ B.T)
        tol[t] = s * ((H / 16 + 16) * 2 * U * ((x.abs() @ A.abs().T) @ B.abs().T) +
                      ((R / 8 + 8) * 2 * U + (2.0 ** -15 if bf16 else 2.0 ** -23)) * (v.abs() @ B.abs().T))
        tol[t] += (2.0 ** -8 if bf16 else U) * out[t].abs() + 1e-30
    return out, tol


def _check(i, out=None):
    want, tol = _reference(i)
    got = eb.lora_add(i["base"], i["x"], i["a"], i["b"], i["adapter_ids"], scales=i["scales"], out=out)
    torch.cuda.synchronize()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    own = (i["adapter_ids"] < 0) | (i["adapter_ids"] >= i["a"].shape[0])
    assert torch.equal(got[own], i["base"][own]) or out is i["base"]
    if got.dtype == torch.float32 and bool((~own).any()):        # typically far inside the worst case
        assert float(err.norm() / want.norm()) < 5e-7
    assert eb.device_status() == 0
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,H,N,R,L", [(1, 8, 8, 8, 1), (1, 8192, 256, 16, 8), (2, 64, 16, 8, 1), (9, 520, 264, 24, 2),
                                       (17, 1032, 40, 16, 3), (33, 2048, 512, 32, 40), (100, 4104, 1000, 40, 7),
                                       (128, 1024, 2048, 128, 16), (255, 512, 128, 64, 5), (256, 512, 72, 96, 4),
                                       (257, 520, 136, 16, 6), (300, 1024, 256, 64, 1), (777, 1536, 520, 48, 9),
                                       (1500, 2048, 2560, 16, 4), (2300, 264, 24, 128, 64),
                                       (300, 64, 16, 8, 1100), (33000, 72, 16, 8, 3), (4500, 64, 24, 16, 1025)])
def test_sizes(cuda_dev, T, H, N, R, L, bf16):
    _check(_inputs(cuda_dev, T, H, N, R, L, bf16, seed=T + H))


@pytest.mark.parametrize("T", [1, 8, 9, 200, 256, 257, 700, 1300])
@pytest.mark.parametrize("kind", ["one", "none", "each", "runs", "outside"])
def test_distributions_of_adapters(cuda_dev, T, kind):
    L = 12
    ids = {"one": [3] * T, "none": [-1] * T, "each": [t % L for t in range(T)], "runs": [t * 5 // T - 1 for t in range(T)],
           "outside": [(-1, 12, 2 ** 31 - 1, -2 ** 31, 4)[t % 5] for t in range(T)]}[kind]
    _check(_inputs(cuda_dev, T, 328, 264, 16, L, T % 2 == 1, seed=T, ids=ids))


@pytest.mark.parametrize("T", [5, 400])
def test_in_place_without_scales_and_guards(cuda_dev, T):
    """out = base; rows without an adapter and memory behind out keep their bits."""
    i = _inputs(cuda_dev, T, 256, 136, 16, 3, False, seed=4)
    i["scales"] = None
    want, tol = _reference(i)
    buf = torch.full((T * 136 + 64,), -7.0, device=cuda_dev)
    y = buf[:T * 136].view(T, 136)
    y.copy_(i["base"])
    assert eb.lora_add(y, i["x"], i["a"], i["b"], i["adapter_ids"], out=y) is y
    torch.cuda.synchronize()
    assert bool(((y.double() - want).abs() <= tol).all()) and bool((buf[T * 136:] == -7).all())
    assert torch.equal(y[i["adapter_ids"] < 0], i["base"][i["adapter_ids"] < 0])


@pytest.mark.parametrize("T,N,R", [(40, 128, 16), (600, 128, 16), (40, 136, 8), (600, 136, 8), (600, 136, 24),
                                   (600, 200, 72)])
def test_unused_values_do_not_leak(cuda_dev, T, N, R):
    """NaN in x of tokens without an adapter, in an adapter nobody uses, and in one token's x stay where they are."""
    ids = [(-1, 0, 2, 2, 0)[t % 5] for t in range(T)]
    i = _inputs(cuda_dev, T, 512, N, R, 4, False, seed=8, ids=ids)
    want, tol = _reference(i)
    i["x"][0::5] = float("nan")
    i["a"][1] = float("nan")
    i["b"][1] = float("inf")
    i["a"][3] = float("inf")
    i["x"][2] = float("nan")
    got = eb.lora_add(i["base"], i["x"], i["a"], i["b"], i["adapter_ids"], scales=i["scales"])
    torch.cuda.synchronize()
    rows = torch.arange(T, device=cuda_dev) != 2
    assert bool(((got.double() - want).abs() <= tol)[rows].all()) and bool(got[2].isnan().all())


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_repeats_bit_for_bit(cuda_dev, T):
    """The same bits on every run, on a side stream and replayed from a graph (with other inputs in the same memory)."""
    i = _inputs(cuda_dev, T, 1024, 520, 32, 6, True, seed=2)
    j = _inputs(cuda_dev, T, 1024, 520, 32, 6, True, seed=3)
    call = lambda k, **kw: eb.lora_add(k["base"], k["x"], k["a"], k["b"], k["adapter_ids"], scales=k["scales"], **kw)  # noqa: E731
    first, other = call(i), call(j)
    again = call(i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = call(i)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, third)
    out = torch.empty_like(first)
    ws = torch.empty(eb.lora_workspace_size(T, 1024, 520, 32, 6), dtype=torch.uint8, device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(i, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    for n in i:
        i[n].copy_(j[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)


@pytest.mark.parametrize("T", [3, 900])
def test_beside_the_router_projection(cuda_dev, T):
    """router_logits, the requests' adapters on its logits in place, and the gate on the sum."""
    H, E, k, L = 1024, 64, 8, 5
    i = _inputs(cuda_dev, T, H, E, 16, L, False, seed=6)
    w = torch.randn(E, H, generator=torch.Generator(device=cuda_dev).manual_seed(1), device=cuda_dev) * H ** -0.5
    logits = eb.router_logits(i["x"], eb.router_weight_prepare(w))
    want, tol = _reference({**i, "base": logits.clone()})
    eb.lora_add(logits, i["x"], i["a"], i["b"], i["adapter_ids"], scales=i["scales"], out=logits)
    ids, weights = eb.moe_route(logits, torch.zeros(E, device=cuda_dev),
                                torch.ones(T, dtype=torch.uint8, device=cuda_dev), k)
    loss, counts, _, n = eb.moe_balance_loss(logits, ids, torch.ones(T, dtype=torch.uint8, device=cuda_dev), 0.1)
    torch.cuda.synchronize()
    assert bool(((logits.double() - want).abs() <= tol).all())
    assert torch.equal(torch.topk(logits, k, dim=1).indices.sort(1).values, ids.long().sort(1).values)
    assert int(n) == T and int(counts.sum()) == T * k and float(loss) > 0


def _shifted(t):
    """The same values at an address that is 16-byte aligned and no more."""
    buf = torch.zeros(t.numel() + 64, dtype=t.dtype, device=t.device)
    step = 16 // t.element_size()
    at = next(k for k in range(step, 64, step) if (buf.data_ptr() + k * t.element_size()) % 32 == 16)
    v = buf[at:at + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("T,bf16", [(30, False), (30, True), (500, False), (500, True)])
def test_addresses_of_16_bytes(cuda_dev, T, bf16):
    i = _inputs(cuda_dev, T, 520, 264, 24, 3, bf16, seed=12)
    _check({k: _shifted(v) for k, v in i.items()}, out=_shifted(i["base"]))


def test_two_streams_at_once(cuda_dev):
    """Calls that overlap on the GPU, each with its own workspace, few and many tokens."""
    cases = [_inputs(cuda_dev, T, 1024, 512, 16, 8, True, seed=T) for T in (64, 2000, 128, 3000)]
    call = lambda i: eb.lora_add(i["base"], i["x"], i["a"], i["b"], i["adapter_ids"], scales=i["scales"])  # noqa: E731
    want = [call(i) for i in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for s, i, g in zip(streams, cases, got):
            with torch.cuda.stream(s):
                g.append(call(i))
    torch.cuda.synchronize()
    assert all(torch.equal(w, x) for w, g in zip(want, got) for x in g)
    assert eb.device_status() == 0


def test_graphs_that_share_a_workspace(cuda_dev):
    """Two captured calls with one workspace, replayed one after the other."""
    i, j = (_inputs(cuda_dev, T, 512, 256, 16, 4, False, seed=T) for T in (700, 900))
    ws = torch.empty(eb.lora_workspace_size(900, 512, 256, 16, 4), dtype=torch.uint8, device=cuda_dev)
    call = lambda k, **kw: eb.lora_add(k["base"], k["x"], k["a"], k["b"], k["adapter_ids"], scales=k["scales"], **kw)  # noqa: E731
    want = [call(i), call(j)]
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for k, o in zip((i, j), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(k, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, o) for w, o in zip(want, outs))


def test_refusals(cuda_dev):
    i = _inputs(cuda_dev, 4, 64, 32, 8, 2, False)
    call = lambda **kw: eb.lora_add(**{**i, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="shape"):
        call(b=i["b"][:, :, :4].contiguous())
    with pytest.raises(ValueError, match="shape"):
        call(adapter_ids=i["adapter_ids"][:3])
    with pytest.raises(ValueError, match="contiguous"):
        call(x=i["x"].t().contiguous().t())
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(scales=i["scales"].cpu())
    with pytest.raises(TypeError, match="expected"):
        call(out=torch.empty(4, 32, dtype=torch.bfloat16, device=cuda_dev))
    with pytest.raises(eb.MoEBoundaryError, match="overlaps"):
        buf = torch.zeros(4 * 32 + 4, device=cuda_dev)
        call(base=buf[:128].view(4, 32), out=buf[4:].view(4, 32))
    with pytest.raises(eb.MoEBoundaryError, match="workspace"):
        eb.lora_add(**_inputs(cuda_dev, 300, 64, 32, 8, 2, False),
                    workspace=torch.empty(16, dtype=torch.uint8, device=cuda_dev))
    with pytest.raises(eb.MoEBoundaryError, match="needs H, N and R"):
        call(a=i["a"][:, :4].contiguous(), b=i["b"][:, :, :4].contiguous())


def _same_class(got, want):
    """NaN where the definition is NaN, an infinity of the definition's sign where it is infinite, else finite."""
    return bool((got.isnan() == want.isnan()).all()) and bool((got.isposinf() == want.isposinf()).all()) and \
        bool((got.isneginf() == want.isneginf()).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,N,R", [(40, 136, 24), (400, 136, 24), (400, 264, 64), (900, 128, 128)])
def test_infinite_values_of_the_second_factor(cuda_dev, T, N, R, bf16):
    """v * inf is an infinity of v's sign, inf - inf and 0 * inf NaN, for few and for many tokens."""
    H, L = 256, 4
    i = _inputs(cuda_dev, T, H, N, R, L, bf16, seed=17)
    inf = float("inf")
    i["b"][1, 5, 3] = inf
    i["b"][1, N - 1, R - 1] = -inf
    i["b"][2, 7, 0], i["b"][2, 7, 1] = inf, -inf
    i["b"][2, 9, 2] = float("nan")
    i["x"][T // 2] = 0.0
    i["x"][T // 3, 10] = inf
    t = torch.nonzero(i["adapter_ids"] >= 0).flatten()
    v = torch.einsum("th,trh->tr", i["x"][t].double(), i["a"][i["adapter_ids"][t].long()].double())
    some = v[v.isfinite() & (v != 0)].abs()
    assert float(some.min()) > 1e-5          # the signs of v are the definition's
    want, tol = _reference(i)
    got = eb.lora_add(i["base"], i["x"], i["a"], i["b"], i["adapter_ids"], scales=i["scales"])
    torch.cuda.synchronize()
    assert _same_class(got, want) and bool(want.isinf().any()) and bool(want.isnan().any())
    ok = want.isfinite()
    assert bool(((got.double() - want).abs() <= tol)[ok].all())
    assert eb.device_status() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [20, 300])
def test_first_products_above_the_largest_bf16(cuda_dev, T, bf16):
    """v between the largest BF16 and the largest FP32 value is no infinity."""
    H, N, R = 64, 16, 8
    i = _inputs(cuda_dev, T, H, N, R, 1, bf16, seed=2, ids=[0] * T)
    for n in ("x", "a", "b"):
        i[n].zero_()
    top = torch.finfo(torch.bfloat16).max
    i["scales"] = None
    i["a"][0, 0, 0] = i["a"][0, 0, 1] = i["a"][0, 1, 2] = i["a"][0, 1, 3] = 1.0
    i["x"][:, 0], i["x"][:, 1], i["x"][:, 2], i["x"][:, 3] = top, 1.5 * 2.0 ** 119, -top, -1.5 * 2.0 ** 119
    i["b"][0, 0, 0], i["b"][0, 1, 1], i["b"][0, 2, 0] = 2.0 ** -100, 2.0 ** -100, 0.5
    want, tol = _reference(i)
    got = eb.lora_add(i["base"], i["x"], i["a"], i["b"], i["adapter_ids"])
    torch.cuda.synchronize()
    assert bool(got.isfinite().all()) and bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T,bf16", [(30, False), (30, True), (500, False), (500, True)])
def test_addresses_of_16_bytes_from_an_empty_output(cuda_dev, T, bf16):
    """Every row is written, also those without an adapter: out holds NaN before the call."""
    i = {k: _shifted(v) for k, v in _inputs(cuda_dev, T, 520, 264, 24, 3, bf16, seed=12).items()}
    out = _shifted(torch.full_like(i["base"], float("nan")))
    assert bool((i["adapter_ids"] < 0).any())
    _check(i, out=out)
