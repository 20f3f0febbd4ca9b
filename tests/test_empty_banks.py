"""Banks of no rows in host memory, whose empty tensors torch cannot pin, and tensors of
too few dimensions."""
import pytest
import torch

import expert_weight_residency_amd as moe

F8 = torch.float8_e4m3fn


def empty_f8(H, I, where, device="cpu"):
    b = (I + 127) // 128, (H + 127) // 128
    return moe.BankF8(torch.zeros(0, 2 * I, H).to(F8), torch.zeros(0, 2, *b, device=device),
                      torch.zeros(0, H, I).to(F8), torch.zeros(0, *b[::-1], device=device), where)


def test_binding_takes_empty_host_banks():
    assert empty_f8(128, 64, moe.BANK_HOST).abi().n_rows == 0
    w = torch.zeros(0, 8, 16).bfloat16()
    assert moe._grouped_weights(w, torch.bfloat16)[1:] == (0, 8, 16, moe.BANK_HOST)
    for bad in (torch.zeros(1, 8, 16).bfloat16(), torch.zeros(0, 8, 16), torch.zeros(0, 8).bfloat16()):
        with pytest.raises(moe.MoeError):
            moe._grouped_weights(bad, torch.bfloat16)
    with pytest.raises(moe.MoeError):  # rows, but not pinned
        moe.BankF8(torch.zeros(1, 128, 128).to(F8), torch.zeros(1, 2, 1, 1), torch.zeros(1, 128, 64).to(F8),
                   torch.zeros(1, 1, 1), moe.BANK_HOST).abi()


@pytest.mark.gpu
def test_a_layer_without_cold_experts():
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    T, k, E, H, I = 5, 2, 3, 128, 64
    g = torch.Generator().manual_seed(1)
    bank = moe.BankF8(torch.randn(E, 2 * I, H, generator=g).to(F8).cuda(), torch.ones(E, 2, 1, 1, device="cuda"),
                      torch.randn(E, H, I, generator=g).to(F8).cuda(), torch.ones(E, 1, 1, device="cuda"))
    rm = torch.arange(E, dtype=torch.int32, device="cuda")
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=g).cuda()
    w, x = torch.rand(T, k, generator=g).cuda(), torch.randn(T, H, generator=g).bfloat16().cuda()
    out = []
    for cold in (empty_f8(H, I, moe.BANK_HOST), empty_f8(H, I, moe.BANK_HOST_WEIGHTS, "cuda"),
                 moe.BankF8(*(t[:0] for t in bank.tensors().values()))):
        layer = ResidencyLayer(bank, cold, rm, H, I)
        bufs = LayerBuffers.allocate(T, k, H, I, E, 0, f8=True)
        layer.forward(x, ids, w, bufs)
        torch.cuda.synchronize()
        out.append(bufs.out.clone())
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[2])
    split = moe.Split.empty(0, T, k)
    y = torch.full((T * k, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear(x, torch.zeros(0, 8, H).bfloat16(), split, k, y)
    dx = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_dx(y, torch.zeros(0, 8, H).bfloat16(), split, k, dx)
    torch.cuda.synchronize()
    assert (y == 7.0).all() and (dx == 7.0).all()


@pytest.mark.gpu
def test_tensors_of_too_few_dimensions():
    T, k, E, N, K = 4, 2, 3, 8, 16
    split = moe.Split.empty(E, T, k)
    bf, dev = torch.bfloat16, "cuda"
    x, w = torch.zeros(T, K, dtype=bf, device=dev), torch.zeros(E, N, K, dtype=bf, device=dev)
    y, dx = torch.zeros(T * k, N, dtype=bf, device=dev), torch.zeros(T * k, K, dtype=bf, device=dev)
    for t in (torch.zeros((), dtype=bf, device=dev), torch.zeros(T * k, dtype=bf, device=dev)):
        for call in (lambda: moe.moe_grouped_linear(x, w, split, k, t), lambda: moe.moe_grouped_linear(t, w, split, k, y),
                     lambda: moe.moe_grouped_linear_dx(t, w, split, k, dx),
                     lambda: moe.moe_grouped_linear_dx(y, w, split, k, t),
                     lambda: moe.moe_grouped_linear_dw(t, x, split, k, w), lambda: moe.moe_grouped_linear_dw(y, t, split, k, w),
                     lambda: moe.moe_grouped_linear_dw(y, x, split, k, t), lambda: moe.moe_grouped_linear(x, t, split, k, y)):
            with pytest.raises(moe.MoeError):
                call()
