"""The gradient of activations that a token's picks share, with padding tokens and picks of
no expert, whose rows of every buffer hold what an earlier step left."""
import pytest
import torch

import expert_weight_residency_amd as moe
from layer_ref import U32, UBF16
from test_gpu_grouped import inputs, make_split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def picks(T, k, E, seed):
    """ids with padding tokens, masked picks and ids outside the map; which of them count."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=g)
    ids[T - T // 5:] = -1
    ids[::3, 1], ids[1, 0], ids[2, k - 1] = -1, E, E + 7
    return ids, (ids >= 0) & (ids < E)


@pytest.mark.parametrize("before", [float("nan"), 3e38, 1000.0])
@pytest.mark.parametrize("T,E,N,K", [(9, 5, 72, 136), (60, 6, 520, 1032), (700, 3, 1032, 264)])
def test_sum_of_the_input_gradient(T, E, N, K, before):
    """moe_finalize with weight 1 for the picks of an expert and 0 for the others, over dx of
    which the others' rows are stale; of two banks, too. The rows are rounded to bf16 once
    (after sums of N products in fp32), the sum of at most k of them once more."""
    k, cold = 3, 2
    ids, ok = picks(T, k, E, T)
    _, dy, w = inputs(T, k, E, N, K, torch.bfloat16, True, 5)
    rows = torch.stack([dy[s].double() @ w[e].double() if ok.view(-1)[s] else torch.zeros(K).double()
                        for s, e in enumerate(ids.view(-1).tolist())]).view(T, k, K)
    size = torch.stack([dy[s].double().abs() @ w[e].double().abs() if ok.view(-1)[s] else torch.zeros(K).double()
                        for s, e in enumerate(ids.view(-1).tolist())]).view(T, k, K)
    off = 2 * N * U32 * size
    off = off + UBF16 * (rows.abs() + off)
    want, tol = rows.sum(1), off.sum(1) + k * U32 * (rows.abs() + off).sum(1)
    tol = tol + UBF16 * (want.abs() + tol) + 2.0 ** -140
    dev = dy.cuda(), w.cuda(), ok.float().cuda()
    for n_cold in (0, cold):
        rm = [e if e < E - n_cold else -1 - (e - (E - n_cold)) for e in range(E)]
        hot, other = make_split(ids, E, rm, n_cold)
        dx = torch.full((T * k, K), before, dtype=torch.bfloat16, device="cuda")
        out = torch.full((T, K), before, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_linear_dx(dev[0], dev[1][:E - n_cold], hot, k, dx)
        if n_cold:
            moe.moe_grouped_linear_dx(dev[0], dev[1][E - n_cold:], other, k, dx)
        moe.moe_finalize(dx, dev[2], out)
        torch.cuda.synchronize()
        err = (out.cpu().double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert (out[T - T // 5:] == 0).all()


def test_a_routed_layer_with_padding_and_its_gradients():
    """The layer of test_gpu_grouped with padding tokens and masked picks, every buffer of
    slots full of NaN before: as there, 5 roundings to bf16 at most on the way to any
    value."""
    T, k, E, H, I = 45, 3, 6, 128, 192
    g = torch.Generator().manual_seed(8)
    ids, ok = picks(T, k, E, 2)
    tw = torch.softmax(torch.randn(T, k, generator=g), 1) * ok
    x = torch.randn(T, H, generator=g).bfloat16()
    w13 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).bfloat16()
    w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).bfloat16()
    dout = torch.randn(T, H, generator=g).bfloat16()
    split, _ = make_split(ids, E)
    S, bf = T * k, torch.bfloat16

    def stale(*shape, dtype=torch.float32):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    xd, ad, bd, twd = x.cuda(), w13.cuda(), w2.cuda(), tw.cuda()
    gu = stale(S, 2 * I)
    moe.moe_grouped_linear(xd, ad, split, k, gu)
    gg, u = gu[:, :I], gu[:, I:]
    sig = torch.sigmoid(gg)
    h = (gg * sig * u).to(bf)
    y, out = stale(S, H, dtype=bf), stale(T, H, dtype=bf)
    moe.moe_grouped_linear(h, bd, split, k, y)
    moe.moe_finalize(y, twd, out)
    dy = (dout.cuda().float().repeat_interleave(k, 0) * twd.reshape(-1, 1)).to(bf)
    dh, dw2 = stale(S, I), stale(E, H, I)
    moe.moe_grouped_linear_dx(dy, bd, split, k, dh)
    moe.moe_grouped_linear_dw(dy, h, split, k, dw2)
    dgu = torch.cat([dh * u * sig * (1 + gg * (1 - sig)), dh * gg * sig], dim=1).to(bf)
    dxs, dw13, dx = stale(S, H, dtype=bf), stale(E, 2 * I, H), stale(T, H, dtype=bf)
    moe.moe_grouped_linear_dx(dgu, ad, split, k, dxs)
    moe.moe_grouped_linear_dw(dgu, xd, split, k, dw13)
    moe.moe_finalize(dxs, ok.float().cuda(), dx)
    torch.cuda.synchronize()

    leaves = [v.double().requires_grad_() for v in (x, w13, w2)]
    at = ids.clamp(0, E - 1).long()
    p = torch.einsum("tkih,th->tki", leaves[1][at], leaves[0])
    hd = torch.nn.functional.silu(p[..., :I]) * p[..., I:]
    ref = (torch.einsum("tkhi,tki->tkh", leaves[2][at], hd) * tw.double().unsqueeze(2)).sum(1)
    grads = torch.autograd.grad((ref * dout.double()).sum(), leaves)
    for name, a, b in zip(("out", "dx", "dw13", "dw2"), (out, dx, dw13, dw2), (ref.detach(), *grads)):
        assert a.isfinite().all(), name
        assert float((a.cpu().double() - b).norm() / b.norm()) <= 5 * 2.0 ** -8, name
