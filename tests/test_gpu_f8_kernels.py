"""Every kernel of the 8-bit floating point products: which calls launch which, each
against the 64-bit form, and results that do not depend on the kernel."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import synth
from f8_ref import blocks
from kernel_instances import held, launched
from test_gpu_f8 import F8, bank_on, check_ffn, check_linear, make_bank, make_linear, quantize, run_ffn

pytestmark = pytest.mark.gpu
NAMES = r"gemm_f8_\w+|quantize_f8"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


# M, N, K, 16-bit outputs, 32-bit outputs
LINEAR = [
    (3, 700, 400, "gemm_f8_tile<32, 32, ", "gemm_f8_tile<32, 32, "),
    (40, 700, 400, "gemm_f8_tile<32, 64, ", "gemm_f8_tile<32, 64, "),
    (300, 3300, 272, "gemm_f8_tile<64, 64, ", "gemm_f8_tile<64, 64, "),
    (700, 3400, 272, "gemm_f8_tile<128, 64, ", "gemm_f8_tile<128, 64, "),
    (1030, 3900, 400, "gemm_f8_big<256, 128, ", "gemm_f8_tile<128, 64, "),
    (1030, 2047, 2064, "gemm_f8_big<128, 128, ", "gemm_f8_tile<128, 64, "),
    (2040, 4090, 144, "gemm_f8_big<256, 128, ", "gemm_f8_tile<128, 64, "),
    (2900, 4000, 528, "gemm_f8_big<256, 192, ", "gemm_f8_tile<128, 64, "),
    (4090, 4080, 272, "gemm_f8_big<256, 256, ", "gemm_f8_tile<128, 64, "),
]
# T, k, E, H, I, gate/up, down
FFN = [
    (9, 2, 5, 320, 192, "gemm_f8_tile<64, 32, 2, 2, 4, true, true", "gemm_f8_tile<64, 32, 2, 2, 4, false, false"),
    (120, 2, 5, 320, 192, "gemm_f8_tile<128, 64, 2, 2, 3, true, true", "gemm_f8_tile<128, 64, 2, 2, 3, false, false"),
]


@pytest.mark.parametrize("M,N,K,k16,k32", LINEAR)
def test_linear_kernels(M, N, K, k16, k32):
    xq, xs, w, ws = make_linear(M, N, K, M + N + K)
    dev = [v.cuda() for v in (xq, xs, w, ws)]
    for dtype, want in ((torch.bfloat16, k16), (torch.float16, k16), (torch.float32, k32)):
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        got = launched(lambda: moe.moe_linear_f8(*dev, y[:M]), NAMES)
        assert len(got) == 1, got
        name = next(iter(got))
        assert name.startswith(want), (want, name)
        if "tile" in name:
            assert name.endswith("true>" if dtype == torch.float32 else "false>"), name
        assert (y[M] == 7.0).all()
        check_linear(y[:M], xq, xs, w, ws)


@pytest.mark.parametrize("T,k,E,H,I,gu,down", FFN)
def test_ffn_kernels(T, k, E, H, I, gu, down):
    b = make_bank(E, H, I, T)
    ids = torch.from_numpy(synth.gaussian_routing(T, k, E, 5)[0].astype(np.int32))
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    bank, none = bank_on(b, "device"), bank_on({n: v[:0] for n, v in b.items()}, "device")
    out = []
    got = launched(lambda: out.append(run_ffn(bank, none, np.arange(E), ids, x, H, I)), NAMES)
    assert any(g.startswith(gu) for g in got) and any(g.startswith(down) for g in got), got
    check_ffn(out[-1], b, ids, x, H, I)


def test_every_kernel_is_launched():
    want = {s for c in LINEAR for s in c[3:]} | {s for c in FFN for s in c[5:]}
    have = held(r"gemm_f8_\w+")
    for h in have:
        assert any(h.startswith(s) for s in want), h
    for s in want:
        assert any(h.startswith(s) for h in have), s
    types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    seen = set()
    for dtype in types:
        for K in (256, 255):  # whole granules, and not
            seen |= launched(lambda: quantize(torch.randn(3, K, device="cuda").to(dtype)), "quantize_f8")
    assert seen == held("quantize_f8") and len(seen) == 6


def test_rows_do_not_depend_on_the_kernel():
    """Rows of a large product, computed again a few at a time, have the same bits; and a
    token's FFN the same in a small step and in a large one."""
    M, N, K = 2900, 4000, 528
    xq, xs, w, ws = (v.cuda() for v in make_linear(M, N, K, 1))
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty(M, N, dtype=dtype, device="cuda")
        moe.moe_linear_f8(xq, xs, w, ws, y)
        for rows in (slice(0, 3), slice(100, 140), slice(700, 1000), slice(2200, 2900)):
            part = torch.empty(rows.stop - rows.start, N, dtype=dtype, device="cuda")
            moe.moe_linear_f8(xq.view(torch.uint8)[rows].contiguous().view(F8), xs[rows].contiguous(), w, ws, part)
            assert torch.equal(part, y[rows]), (dtype, rows)
    T, k, E, H, I = 200, 2, 5, 320, 192
    b = make_bank(E, H, I, T)
    ids = torch.from_numpy(synth.gaussian_routing(T, k, E, 5)[0].astype(np.int32))
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    bank, none = bank_on(b, "device"), bank_on({n: v[:0] for n, v in b.items()}, "device")
    Y = run_ffn(bank, none, np.arange(E), ids, x, H, I)
    for at in range(0, T, 20):
        part = run_ffn(bank, none, np.arange(E), ids[at:at + 20], x[at:at + 20], H, I)
        assert torch.equal(part.view(torch.int16), Y[at * k:(at + 20) * k].view(torch.int16))


def test_wide_tiles_strides_and_partial_blocks():
    """Large products with strided activations and outputs, and widths that end inside a
    block and a tile."""
    for M, N, K in ((2900, 4000, 528), (4090, 4080, 272), (2040, 4090, 144), (1030, 3900, 400)):
        xq, xs, w, ws = make_linear(M, N, K, 3)
        wide = torch.full((M, K + 32), 0x7f, dtype=torch.uint8, device="cuda").view(F8)
        wide.view(torch.uint8)[:, 16:16 + K] = xq.cuda().view(torch.uint8)
        big = torch.full((M, N + 7), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_linear_f8(wide[:, 16:16 + K], xs.cuda(), w.cuda(), ws.cuda(), big[:, 3:3 + N])
        torch.cuda.synchronize()
        check_linear(big[:, 3:3 + N], xq, xs, w, ws)
        assert (big[:, :3] == 7.0).all() and (big[:, 3 + N:] == 7.0).all()
        assert xs.shape == (M, blocks(K))
