"""Every kernel instance of the few-token layer, the router's gate and the row
quantisation: sizes that reach those no other test does, and that the sizes here
reach every instance the library holds."""
import pytest
import torch

import expert_weight_residency_amd as moe
import layer_ref
import test_gpu_gate
import test_gpu_i8
from kernel_instances import held, launched
from test_gpu_layer_few import check, make_step, row_of, run

pytestmark = pytest.mark.gpu

# (H, I) -> gate/up's chunks per wavefront, ring slots, whole slices; down's chunks per wavefront
AXES = {(320, 3200): ("1, {}, 4, false", 4), (2112, 1088): ("2, {}, 2, false", 2),
        (4096, 576): ("2, {}, 2, true", 1), (4160, 2112): ("4, {}, 2, false", 3),
        (8192, 192): ("4, {}, 2, true", 1), (64, 4096): ("1, {}, 4, false", 4)}
TOKENS = (5, 9)  # one set of columns, two
GATE = {(6, 40, 5): 1, (5, 100, 3): 2, (9, 200, 7): 4, (4, 384, 6): 6, (3, 500, 8): 8, (7, 900, 9): 16,
        (2, 1800, 32): 32, (4, 4001, 2): 64}  # T, E, k -> logits per lane
QUANT = {512: "64, 1", 1992: "256, 1", 2880: "256, 2", 8192: "256, 4", 100: "256, 0", 8200: "256, 0"}
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def step(T, H, I):
    return make_step(T, 3, 7, H, I, 3, T + H)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H,I", list(AXES))
def test_few(T, H, I):
    """Against 64 bits, and the same bits with the cold experts on the host."""
    rm, arr, ids, w, x = step(T, H, I)
    out, ninv = run(arr, rm, ids, w, x, H, I)
    ref, bound, bad = layer_ref.layer(arr, row_of(rm, 4, 3), x, ids, w, H, I)
    assert ninv == bad == 0
    check(out, ref, bound)
    host, _ = run(arr, rm, ids, w, x, H, I, ("device", "host"))
    assert torch.equal(host.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("T,E,k", list(GATE))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gate(T, E, k, dtype):
    l = (torch.randn(T, E, generator=torch.Generator().manual_seed(E)) * 3).to(dtype)
    l[T - 1, k // 2:] = float("nan")
    for norm in (moe.GATE_NORM_PICKS, moe.GATE_NORM_ALL):
        test_gpu_gate.check(l.cuda(), k, norm)


@pytest.mark.parametrize("K", list(QUANT))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_quantize(K, dtype):
    x = torch.randn(6, K, generator=torch.Generator().manual_seed(K))
    test_gpu_i8.check_quantize((x * torch.logspace(-3, 3, 6)[:, None]).to(dtype).cuda())


def test_the_sizes_reach_every_instance():
    reached = set()
    for (H, I), (gate_up, down) in AXES.items():
        for T in TOKENS:
            sets = 1 if T <= 8 else 2
            rm, arr, ids, w, x = step(T, H, I)
            for where in ("device", "host"):
                got = launched(lambda: run(arr, rm, ids, w, x, H, I, ("device", where)), "few_[a-z_]+")
                assert got == {f"few_gate_up<{gate_up.format(sets)}>",
                               f"few_down<{down}, {sets}, {'true' if where == 'host' else 'false'}>"}, (T, H, I)
                reached |= got
    for (T, E, k), per in GATE.items():
        l = torch.randn(T, E, device="cuda")
        got = launched(lambda: test_gpu_gate.gate(l, k, moe.GATE_NORM_ALL), "topk_gate")
        assert got == {f"topk_gate<{per}>"}, (T, E, k)
        reached |= got
    for K, shape in QUANT.items():
        for dtype, code in TYPES.items():
            x = torch.randn(6, K, device="cuda").to(dtype)
            got = launched(lambda: test_gpu_i8.quantize(x), "quantize_rows")
            assert got == {f"quantize_rows<{code}, {shape}>"}, (K, dtype)
            reached |= got
    every = held("few_[a-z_]+|topk_gate|quantize_rows")
    assert reached == every, reached ^ every
