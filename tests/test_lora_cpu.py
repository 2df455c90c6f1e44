"""lora_add without a GPU: the refusals of the library and the binding."""
import ctypes

import pytest
import torch

import expert_combine_b200 as eb

BF16, I32 = torch.bfloat16, torch.int32


def test_host_tensors_and_wrong_types_are_refused():
    T, H, N, R, L = 4, 64, 32, 8, 2
    rest = (torch.zeros(T, H, dtype=BF16), torch.zeros(L, R, H, dtype=BF16), torch.zeros(L, N, R, dtype=BF16),
            torch.zeros(T, dtype=I32))
    for dt in (torch.float32, BF16):
        with pytest.raises(ValueError, match="CUDA tensor"):
            eb.lora_add(torch.zeros(T, N, dtype=dt), *rest)
    for dt in (torch.float16, torch.float64):
        with pytest.raises(TypeError, match="expected"):
            eb.lora_add(torch.zeros(T, N, dtype=dt), *rest)


def test_library_refuses_before_any_launch():
    lib = eb.load()
    base, x, a, b, ids, out, ws = (ctypes.c_void_p(i << 32) for i in range(1, 8))
    odd, N0 = ctypes.c_void_p((1 << 32) + 8), None

    def call(base=base, bf16=0, x=x, T=4, H=64, a=a, b=b, N=32, R=8, L=2, ids=ids, scales=None, out=out, ws=ws,
             size=1 << 40):
        return lib.lora_add(base, bf16, x, T, H, a, b, N, R, L, ids, scales, out, ws, ctypes.c_size_t(size), None)
    assert call(T=0) == 0                                     # empty: no launch
    assert call(T=-1) == 1 and call(L=-1) == 1 and call(bf16=2) == 1
    for bad in (dict(H=4), dict(H=60), dict(H=65544), dict(N=0), dict(N=12), dict(N=262152), dict(R=0), dict(R=12),
                dict(R=136), dict(L=0), dict(L=4097), dict(T=(1 << 24) + 1)):
        assert call(**bad) == 2, bad
    for name in ("base", "x", "a", "b", "ids", "out"):
        assert call(**{name: N0}) == 1 and "null" in eb.last_error()
        assert call(**{name: odd}) == 1 and "aligned" in eb.last_error()
    assert call(scales=odd) == 1
    assert eb.lora_workspace_size(4, 64, 32, 8, 2) == 0       # few tokens need none
    assert call(T=300, ws=N0) == 1 and "workspace" in eb.last_error()
    need = eb.lora_workspace_size(300, 64, 32, 8, 2)
    assert need > 0 and call(T=300, size=need - 1) == 1 and call(T=300, ws=odd) == 1
    # out is base itself or apart from every input
    shifted = ctypes.c_void_p((1 << 32) + 16)
    assert call(out=shifted) == 1 and "overlaps" in eb.last_error()
    for name, p in (("x", x), ("a", a), ("b", b), ("ids", ids)):
        assert call(out=p) == 1 and "overlaps" in eb.last_error(), name
    assert call(scales=out) == 1 and "overlaps" in eb.last_error()
    assert call(T=300, ws=out) == 1 and call(T=300, ws=base) == 1 and "workspace overlaps" in eb.last_error()
    assert eb.lora_workspace_size(4, 64, 32, 9, 2) == 0
    assert eb.supported(eb.STAGE_LORA, 1, 8192, 256, 16, 8) and not eb.supported(eb.STAGE_LORA, 1, 8192, 256, 256, 8)
    assert not eb.supported(eb.STAGE_LORA, 1, 64, 262144, 8, 4097)


def test_workspace_over_any_array_is_refused():
    """The plan and the partial sums of a batch may share no byte with what the call reads."""
    lib = eb.load()
    T, H, N, R, L = 300, 64, 32, 8, 2
    need = eb.lora_workspace_size(T, H, N, R, L)
    size = {"base": T * N * 4, "x": T * H * 2, "a": L * R * H * 2, "b": L * N * R * 2, "ids": T * 4, "scales": L * 4,
            "out": T * N * 4}
    at = {n: (i + 1) << 32 for i, n in enumerate(size)}
    P = {n: ctypes.c_void_p(a) for n, a in at.items()}
    for n in size:
        for ws in (at[n], (at[n] + size[n] - 1) & ~255, at[n] - ((need - 1) & ~255)):
            assert lib.lora_add(P["base"], 0, P["x"], T, H, P["a"], P["b"], N, R, L, P["ids"], P["scales"], P["out"],
                                ctypes.c_void_p(ws), ctypes.c_size_t(need), None) == 1, n
            assert "workspace overlaps" in eb.last_error(), n
