"""The 8-bit floating point products sum in 32 bits, whatever their output's type: against
the 64-bit form with no slack but fp32's own and the output's rounding, on inputs where a
few products are far larger than the rest; and special values, in every kernel of the
dense product and of the expert FFN."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import f8_ref
from f8_ref import blocks
from kernel_instances import launched
from layer_ref import HALF_STEP
from test_gpu_f8 import F8, TYPES, bank_on, make_linear, run_ffn
from test_gpu_f8_kernels import LINEAR, NAMES

pytestmark = pytest.mark.gpu
SIZES = [c[:4] for c in LINEAR]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def linear(xq, xs, w, ws, dtype, kernel=None):
    M, N = xq.shape[0], w.shape[0]
    dev = [v.cuda() for v in (xq, xs, w, ws)]
    y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
    if kernel is None:
        moe.moe_linear_f8(*dev, y[:M])
    else:
        got = launched(lambda: moe.moe_linear_f8(*dev, y[:M]), NAMES)
        assert len(got) == 1 and next(iter(got)).startswith(kernel), got
    assert (y[M] == 7.0).all()
    return y[:M]


def check_sums(y, xq, xs, w, ws):
    """fp32's bound (f8_ref.product's for a 32-bit output) and one rounding to y's type."""
    ref, off = f8_ref.product(f8_ref.values(xq), xs, f8_ref.values(w), ws, torch.float32)
    tiny = 2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -140
    tol = off + HALF_STEP[y.dtype] * (ref.abs() + off) + tiny
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_outliers(M, N, K, kernel):
    """Two products of 448 * 448 in each block, of opposite signs and 8 elements apart, among
    products of about 8: what is left is the others' sum, which a sum that cuts them at
    2^-13 of the largest product beside them would lose."""
    g = torch.Generator().manual_seed(M + N)
    x = (torch.randn(M, K, generator=g) * 2).clamp(-4, 4)
    w = (torch.randn(N, K, generator=g) * 4).clamp(-16, 16)
    x[:, ::128], x[:, 8::128], w[:, ::128], w[:, 8::128] = 448, -448, 448, 448
    xs = torch.rand(M, blocks(K), generator=g) + 0.5
    ws = (torch.rand(blocks(N), blocks(K), generator=g) + 0.5) / 16
    xq, w = x.to(F8), w.to(F8)
    for dtype in TYPES:
        check_sums(linear(xq, xs, w, ws, dtype, kernel if dtype != torch.float32 else None), xq, xs, w, ws)


@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_large_products_that_cancel(M, N, K, kernel):
    """448 * 448 - 448 * 448 + 6 * 15 in each run of 8 elements: 90, or what is left of the
    15s where the row ends. The sums are whole numbers below 2^24 and so is every part of
    them: exact in fp32, and then rounded once."""
    a, b = torch.full((M, K), 15.0), torch.ones(N, K)
    a[:, ::8], a[:, 1::8] = 448, -448
    b[:, ::8], b[:, 1::8] = 448, 448
    b[1::2] = -b[1::2]
    xs, ws = torch.ones(M, blocks(K)), torch.full((blocks(N), blocks(K)), 2.0 ** -4)
    want = torch.full((M, N), 90.0 * (K // 8) / 16)
    want[:, 1::2] *= -1
    for dtype in TYPES:
        y = linear(a.to(F8), xs, b.to(F8), ws, dtype, kernel if dtype != torch.float32 else None)
        assert torch.equal(y.cpu(), want.to(dtype)), dtype


@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_types_round_the_same_sums(M, N, K, kernel):
    """16-bit outputs are the 32-bit ones, rounded; and rows taken a few at a time, by other
    kernels, have the same bits."""
    xq, xs, w, ws = make_linear(M, N, K, M + K)
    wide = linear(xq, xs, w, ws, torch.float32)
    dev = [v.cuda() for v in (xq, xs, w, ws)]
    for dtype in TYPES[:2]:
        y = linear(xq, xs, w, ws, dtype, kernel)
        assert torch.equal(y, wide.to(dtype)), dtype
        for rows in (slice(0, 3), slice(M // 2, M // 2 + 40), slice(M - min(M, 700), M)):
            part = torch.empty(y[rows].shape, dtype=dtype, device="cuda")
            moe.moe_linear_f8(dev[0].view(torch.uint8)[rows].contiguous().view(F8), dev[1][rows].contiguous(),
                              dev[2], dev[3], part)
            assert torch.equal(part, y[rows]), (dtype, rows)


def test_every_block_of_a_long_sum_counts():
    """Positive codes, so that each of the 1024 blocks is about 1/1024 of the sum: more than
    the bound of fp16 outputs, a half step of 2^-11 and fp32's (256 + 2048 + 2) 2^-24."""
    M, N, K = 5, 3, 131072
    g = torch.Generator().manual_seed(1)
    xq, w = ((torch.rand(s, K, generator=g) + 0.5).to(F8) for s in (M, N))
    xs, ws = torch.ones(M, blocks(K)), torch.full((1, blocks(K)), 2.0 ** -4)
    for dtype in TYPES:
        check_sums(linear(xq, xs, w, ws, dtype), xq, xs, w, ws)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_special_values(M, N, K, kernel, dtype):
    """A NaN code or scale reaches the outputs that read it and no others, in the first, a
    middle and the last rows and blocks; an infinite scale of the last, part-filled block
    gives infinities."""
    xq, xs, w, ws = make_linear(M, N, K, 9)
    last, tail = blocks(K) - 1, 128 * (blocks(K) - 1)
    xq.view(torch.uint8)[:, tail:] = 0x38  # 1.0
    w.view(torch.uint8)[:, tail:] = 0x38
    name = kernel if dtype != torch.float32 else None
    base = linear(xq, xs, w, ws, dtype, name)
    assert base.isfinite().all()
    bad_x, bad_xs, bad_w, bad_ws = xq.clone(), xs.clone(), w.clone(), ws.clone()
    bad_w.view(torch.uint8)[5, 130] = 0x7f
    bad_w.view(torch.uint8)[N // 2, K - 1] = 0xff
    bad_ws[blocks(N) - 1, last] = float("inf")
    bad_x.view(torch.uint8)[0, 3] = 0xff
    bad_x.view(torch.uint8)[M // 2, K - 1] = 0x7f
    if M > 3:
        bad_xs[M - 1, last] = float("nan")
    y = linear(bad_x, bad_xs, bad_w, bad_ws, dtype, name)
    rows = {0, M // 2} | ({M - 1} if M > 3 else set())
    edge = 128 * (blocks(N) - 1)
    keep_m = torch.tensor([m for m in range(M) if m not in rows], device="cuda")
    keep_n = torch.tensor([n for n in range(edge) if n not in (5, N // 2)], device="cuda")
    assert y[list(rows)].isnan().all() and y[:, 5].isnan().all() and y[:, N // 2].isnan().all()
    assert torch.equal(y[keep_m][:, keep_n], base[keep_m][:, keep_n])
    assert (y[keep_m][:, [n for n in range(edge, N) if n != N // 2]] == float("inf")).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantised_special_blocks(dtype):
    """Rows with zeros, an infinity, a NaN and subnormal scales, quantised and multiplied."""
    for M in (7, 1030):
        x = torch.randn(M, 256, generator=torch.Generator().manual_seed(6))
        x[0, :128] = 0.0
        x[1, 5] = float("inf")
        x[2, 255] = float("nan")
        x[3, 128:] *= 1e-40
        x[5] = -0.0
        q = torch.empty(M, 256, dtype=F8, device="cuda")
        s = torch.empty(M, 2, device="cuda")
        moe.moe_quantize_rows_f8(x.cuda(), q, s)
        w, ws = torch.ones(3900, 256).to(F8), torch.ones(31, 2)
        y = linear(q.cpu(), s.cpu(), w, ws, dtype)
        assert y[[1, 2]].isnan().all() and (y[5] == 0).all()
        rest = [m for m in range(M) if m not in (1, 2)]
        assert y[rest].isfinite().all()
        check_sums(y[rest], q.cpu().view(torch.uint8)[rest].view(F8), s.cpu()[rest], w, ws)


@pytest.mark.parametrize("T", [9, 120])
def test_ffn_down_product_of_cancelling_rows(T):
    """Experts whose gate is 64 before the activation, so that h is exactly 64 times up's
    values, which are codes with 448 in every block: the down products cancel as above, in
    either of the two kernels. 12845056 = 28672 * 448 is h's scale, exactly."""
    k, E, H, I = 2, 3, 192, 320
    up = torch.full((I,), 15.0)
    up[::8], up[1::8] = 448, -448
    w13 = torch.zeros(E, 2 * I, H)
    w13[:, :I, 0] = 64   # gate: 448 * 64
    w13[:, I:, 0] = up   # 448 * up
    w2 = torch.ones(E, H, I)
    w2[:, :, ::8], w2[:, :, 1::8] = 448, 448
    w2[:, 1::2] *= -1
    b = {"w13": w13.to(F8), "w2": w2.to(F8), "s13": torch.ones(E, 2, blocks(I), blocks(H)),
         "s2": torch.full((E, blocks(H), blocks(I)), 2.0 ** -20)}
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 448
    x[1] = 0
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    none = {n: v[:0] for n, v in b.items()}
    hot, cold, out = bank_on(b, "device"), bank_on(none, "device"), []
    got = launched(lambda: out.append(run_ffn(hot, cold, np.arange(E), ids, x, H, I)), r"gemm_f8_\w+")
    assert any(g.startswith("gemm_f8_tile<64" if T < 16 else "gemm_f8_tile<128") for g in got), got
    want = torch.full((T, k, H), 90.0 * (I // 8) * 12.25)
    want[:, :, 1::2] *= -1
    want[1] = 0
    assert torch.equal(out[-1].view(T, k, H), want.bfloat16())
