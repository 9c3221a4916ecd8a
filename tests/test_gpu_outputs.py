"""GPU: tensors that the calls allocate come the way torch's own do: filled where
torch fills uninitialised memory, and seen by dispatch modes."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu


@pytest.fixture
def deterministic():
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(before)


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.sizes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket is torch.ops.aten.empty:
            self.sizes.append(tuple(args[0]))
        return func(*args, **(kwargs or {}))


def layer_calls(lib):
    """(name, call, sizes that it allocates) of the operators around attention."""
    codes, words = torch.zeros(4, 512, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    w, ws = torch.zeros(256, 512, dtype=torch.uint8, device="cuda"), torch.zeros(2, 4, dtype=torch.uint8, device="cuda")
    q, k = (torch.zeros(4, h, 128, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    cache = lib.fp8_kv_cache(4, 1, head_dim=128, block_size=16, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens, cu = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    return [
        ("product", lambda: lib.fp8_gemm_1x128_128x128(codes, words, w, ws), [(4, 256)]),
        ("attention", lambda: lib.attention_fp8_kv(q, cache, table, lens, cu), [(4, 2, 128)]),
    ]


def moe_calls(lib):
    index = torch.tensor([[0, 1], [1, -1], [2, 2]], dtype=torch.int32, device="cuda")
    groups = lib.group_rows(index, 2)
    codes, words = torch.zeros(3, 256, dtype=torch.uint8, device="cuda"), torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w, ws = torch.zeros(2, 256, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 2, 2, dtype=torch.uint8, device="cuda")
    y = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    return [
        ("route", lambda: lib.moe_route(torch.ones(3, 8, device="cuda"), 2), [(3, 2), (3, 2)]),
        ("group", lambda: lib.group_rows(index, 2), [(3,), (6,), (3, 2)]),
        ("product", lambda: lib.fp8_grouped_gemm_1x128_128x128(codes, words, w, ws, groups, gather=True), [(6, 256)]),
        ("swiglu", lambda: lib.fp8_grouped_swiglu_1x128(codes, words, w, ws, groups, gather=True), [(6, 128), (6, 1)]),
        ("combine", lambda: lib.moe_combine(y, groups, torch.ones(3, 2, device="cuda")), [(3, 64)]),
    ]


def test_dispatch_modes_see_the_allocations(gpu_lib):
    for name, call, sizes in layer_calls(gpu_lib) + moe_calls(gpu_lib):
        print("allocations", name, flush=True)
        with Allocations() as seen:
            call()
        assert all(s in seen.sizes for s in sizes), (name, seen.sizes)


def test_uninitialised_memory_is_filled(gpu_lib, deterministic):
    """With deterministic algorithms torch fills what no kernel writes: NaN, or an
    integer type's largest value."""
    calls = {name: call for name, call, _ in moe_calls(gpu_lib)}
    out = calls["product"]()
    assert not bool(torch.isnan(out[:3].float()).any()) and bool(torch.isnan(out[3:].float()).all())
    q, words = calls["swiglu"]()
    assert bool((q[3:] == 255).all()) and bool((words[3:] == (1 << 31) - 1).all()) and bool((q[:3] == 0).all())


def test_rows_of_no_sequence_are_filled(gpu_lib, deterministic):
    calls = {name: call for name, call, _ in layer_calls(gpu_lib)}
    out = calls["attention"]()
    assert bool(torch.isnan(out[3:].float()).all()) and not bool(torch.isnan(out[:3].float()).any())
