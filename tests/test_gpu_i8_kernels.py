"""Every kernel instance behind the 8-bit products, at ragged sizes with enough
steps to turn its buffers over: the dense product and the expert FFN against
exact integer sums in 64 bits, and that the sizes here reach every instance the
library holds (a moved threshold must not leave one untested)."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
from kernel_instances import held, launched
from layer_ref import HALF_STEP, U32
from test_gpu_i8 import check_ffn, make_bank, run_ffn, bank_on

pytestmark = pytest.mark.gpu

KERNELS = "gemm_i8_[a-z]+"

# Tiles. 128-byte steps of K that are no multiple of the buffers, a part-filled
# last step, part-filled last tiles, a last group of fewer than 8 rows of tiles.
TILES = {
    (5043, 6300, 528): "gemm_i8_big<256, 256, 2>",
    (4096, 4095, 1040): "gemm_i8_big<256, 256, 2>",
    (5043, 3300, 656): "gemm_i8_big<192, 256, 2>",
    (4000, 5700, 912): "gemm_i8_big<192, 256, 2>",
    (5043, 3137, 1168): "gemm_i8_big<128, 256, 3>",
    (500, 4096, 4096): "gemm_i8_big<128, 128, 3>",
    (385, 4100, 2064): "gemm_i8_big<128, 128, 3>",
    (1200, 1700, 2192): "gemm_i8_big<128, 128, 3>",
    (1001, 2047, 1040): "gemm_i8_tile<128, 64, 4, 2, 3, false>",
    (700, 1600, 1168): "gemm_i8_tile<64, 64, 2, 2, 3, false>",
    (641, 1665, 400): "gemm_i8_tile<64, 64, 2, 2, 3, false>",
    (112, 1000, 2896): "gemm_i8_tile<32, 64, 2, 2, 4, false>",
    (17, 63, 9232): "gemm_i8_tile<32, 64, 2, 2, 4, false>",
}
# Few rows times few long ones, or many of 4096 or 8192: chunks of 128 bytes per
# wavefront; rows of whole lines and not.
STREAM = {(M, N, K): f"gemm_i8_stream<{4 if K == 4096 else 8}, {1 if M <= 8 else 2}, {'false' if K % 128 else 'true'}>"
          for N, K in ((16391, 4096), (16391, 8192), (45, 8192), (1030, 7056), (2047, 6160)) for M in (1, 7, 12)}
# Few rows elsewhere
FEW = {(M, 45, K): "gemm_i8_tile<32, 64, 2, 2, 4, false>" for K in (1008, 1024, 2048, 2896, 4096, 5136)
       for M in (1, 12)}
FEW[(5, 16421, 1936)] = "gemm_i8_tile<64, 64, 2, 2, 3, false>"
FEW[(16, 33001, 1936)] = "gemm_i8_tile<128, 64, 4, 2, 3, false>"
FEW.update({(M, N, K): "gemm_i8_tile<128, 64, 4, 2, 3, false>"
            for M, N, K in ((16, 33001, 4112), (64, 33001, 2064), (17, 66000, 272), (3, 40001, 7184))})
FEW[(65, 16390, 2064)] = "gemm_i8_big<128, 128, 3>"
# Expert FFN, gate/up (K = H) and down (K = I): T, k, E, H, I
FFN = [(4, 2, 3, H, 192) for H in (960, 1024, 1984, 2048, 2880, 2944, 4032, 4096, 5120, 5184, 7104, 8192)]
FFN += [(3, 2, 3, 128, 5184), (90, 3, 5, 1088, 320), (90, 3, 5, 320, 1088)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def linear(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N * 3 + K)
    xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xq[0], w[N - 1] = 127, -128
    xs = torch.rand(M, device="cuda", generator=g) + 0.01
    ws = torch.rand(N, device="cuda", generator=g) / (73 * K ** 0.5)
    return xq, xs, w, ws


@pytest.mark.parametrize("M,N,K", list(TILES) + list(STREAM) + list(FEW))
def test_dense(M, N, K):
    xq, xs, w, ws = linear(M, N, K)
    # sums of integers below 2^53: exact in any order
    ref = (xq.double() @ w.double().T.contiguous()) * xs.double()[:, None] * ws.double()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        moe.moe_linear_i8(xq, xs, w, ws, y[:M])
        torch.cuda.synchronize()
        assert (y[M] == 7.0).all()
        # the sum to fp32, two products, the type's rounding (and fp16's subnormals)
        tol = (3.1 * U32 + HALF_STEP[dtype]) * ref.abs() + (2.0 ** -25 if dtype == torch.float16
                                                           else 2.0 ** -140)
        off = (y[:M].double() - ref).abs()
        assert bool((off <= tol).all()), (dtype, float((off / tol).max()))


def ffn_step(T, k, E, H, I):
    b = make_bank(E, H, I, T + E + H)
    g = torch.Generator().manual_seed(H + I)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    return b, ids, x


def run(b, ids, x, H, I):
    none = {n: v[:0] for n, v in b.items()}
    return run_ffn(bank_on(b, "device"), bank_on(none, "device"), np.arange(len(b["s2"])), ids, x, H, I)


@pytest.mark.parametrize("T,k,E,H,I", FFN)
def test_expert_ffn(T, k, E, H, I):
    b, ids, x = ffn_step(T, k, E, H, I)
    check_ffn(run(b, ids, x, H, I), b, ids, x, H, I)


def test_the_sizes_reach_every_instance():
    """Which instance a size selects is the dispatch rules' choice on a card of
    256 CUs."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
    reached = set()
    for (M, N, K), want in {**TILES, **STREAM, **FEW}.items():
        xq, xs, w, ws = linear(M, N, K)
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        got = launched(lambda: moe.moe_linear_i8(xq, xs, w, ws, y), KERNELS)
        assert got == {want}, (M, N, K, got)
        reached |= got
    for M in (1, 16):  # weights off a line
        xq, xs, w, ws = linear(M, 16391, 4096)
        off = torch.empty(w.numel() + 16, dtype=torch.int8, device="cuda")[16:].view(w.shape)
        y, z = (torch.empty(M, 16391, device="cuda") for _ in range(2))
        got = launched(lambda: moe.moe_linear_i8(xq, xs, off.copy_(w), ws, y), KERNELS)
        assert got == {f"gemm_i8_stream<4, {1 if M <= 8 else 2}, false>"}, got
        moe.moe_linear_i8(xq, xs, w, ws, z)
        assert torch.equal(y, z)
        reached |= got
    for shape in FFN:
        got = launched(lambda: run(*ffn_step(*shape), *shape[3:]), KERNELS)
        assert got == {f"gemm_i8_tile<128, 64, 4, 2, 3, {gu}>" for gu in ("true", "false")}, (shape, got)
        reached |= got
    assert reached == held(KERNELS), held(KERNELS) ^ reached
