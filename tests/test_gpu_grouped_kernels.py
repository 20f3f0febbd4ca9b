"""Every kernel of the products grouped by expert: which calls launch which, and that the
forward product and the input's gradient give the same bits whichever does."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import synth
from kernel_instances import held, launched
from test_gpu_grouped import check, inputs, make_split, routing, run

pytestmark = pytest.mark.gpu
NAMES = r"grouped\w*"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


# sizes on both sides of each rule, each call's kernel by the start of its name
# T, k, E, N, K, forward, input, weights
SIZES = [
    (40, 2, 6, 72, 136, "grouped<0, {}, 64", "grouped<1, {}, 64", "grouped<2, {}, 64"),
    (300, 2, 60, 1304, 1400, "grouped<0, {}, 128", "grouped<1, {}, 128", "grouped_gradient<2, {}>"),
    (1600, 2, 4, 4096, 1032, "grouped_forward<{}>", "grouped<1, {}, 128", "grouped_gradient<2, {}>"),
    (1500, 2, 4, 264, 5000, "grouped<0, {}, 64", "grouped_gradient<1, {}>", "grouped<2, {}, 64"),
    (100, 2, 4, 1032, 1800, "grouped<0, {}, 64", "grouped<1, {}, 64", "grouped<2, {}, 128"),
    (700, 3, 7, 2600, 2056, "grouped<0, {}, 128", "grouped<1, {}, 128", "grouped_gradient<2, {}>"),
    (300, 2, 6, 16, 1032, "grouped_narrow<{}, 1>", "grouped<1, {}, 64", "grouped<2, {}, 64"),
    (200, 2, 5, 32, 520, "grouped_narrow<{}, 2>", "grouped<1, {}, 64", "grouped<2, {}, 64"),
    (900, 2, 5, 4104, 48, "grouped_short<{}>", "grouped<1, {}, 64", "grouped<2, {}, 64"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,E,N,K,fwd,inp,wts", SIZES)
def test_kernels(T, k, E, N, K, fwd, inp, wts, dtype):
    ids = routing(T, k, E)
    ids[3] = -1
    split, _ = make_split(ids, E)
    code = {torch.bfloat16: 0, torch.float16: 1}[dtype]
    for by_token, out, grad in ((True, dtype, torch.float32), (False, torch.float32, dtype)):
        x, dy, w = inputs(T, k, E, N, K, dtype, by_token, 3)
        dev = [v.cuda() for v in (x, dy, w)]
        y, dx, dw = run(*dev, split, k, out, grad)
        check(ids, x, dy, w, y, dx, dw)
    for want, call in ((fwd, lambda: moe.moe_grouped_linear(dev[0], dev[2], split, k, y)),
                       (inp, lambda: moe.moe_grouped_linear_dx(dev[1], dev[2], split, k, dx)),
                       (wts, lambda: moe.moe_grouped_linear_dw(dev[1], dev[0], split, k, dw))):
        got = launched(call, NAMES)
        assert len(got) == 1 and next(iter(got)).startswith(want.format(code)), (want, got)


def test_every_kernel_is_launched():
    """The kernels that the library holds are those that test_kernels names, for both types."""
    start = {s[i].format(code) for s in SIZES for i in (5, 6, 7) for code in (0, 1)}
    have = held(NAMES)
    assert len(have) == len(start)
    for h in have:
        assert any(h.startswith(s) for s in start), h


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_bits_do_not_depend_on_banks_or_kernel(out):
    """Two experts with most rows in one bank, the others in another, against all in one
    (wide tiles), and the step cut into parts (small ones)."""
    T, k, E, N, K = 1500, 2, 8, 4096, 5128
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(0, 2, (T, k), dtype=torch.int32, generator=g)
    ids[:60] = torch.randint(2, E, (60, k), dtype=torch.int32, generator=g)
    x, dy, w = (v.cuda() for v in inputs(T, k, E, N, K, torch.bfloat16, True, 5))
    one, _ = make_split(ids, E)
    y = torch.full((T * k, N), 7.0, dtype=out, device="cuda")
    dx = torch.full((T * k, K), 7.0, dtype=out, device="cuda")
    moe.moe_grouped_linear(x, w, one, k, y)
    moe.moe_grouped_linear_dx(dy, w, one, k, dx)
    rm = np.array([0, 1] + [-1 - i for i in range(E - 2)], dtype=np.int32)
    hot, cold = make_split(ids, E, rm, E - 2)
    y2, dx2 = torch.full_like(y, 7.0), torch.full_like(dx, 7.0)
    kernels = set()
    for split, part in ((hot, w[:2].contiguous()), (cold, w[2:].contiguous())):
        kernels |= launched(lambda: moe.moe_grouped_linear(x, part, split, k, y2), NAMES)
        kernels |= launched(lambda: moe.moe_grouped_linear_dx(dy, part, split, k, dx2), NAMES)
    assert torch.equal(y, y2) and torch.equal(dx, dx2)
    for at in range(0, T, 30):  # 30 tokens at a time
        rows = slice(at, at + 30)
        part, _ = make_split(ids[rows], E)
        ys = torch.full((30 * k, N), 7.0, dtype=out, device="cuda")
        dxs = torch.full((30 * k, K), 7.0, dtype=out, device="cuda")
        def call():
            moe.moe_grouped_linear(x[rows], w, part, k, ys)
            moe.moe_grouped_linear_dx(dy[at * k:(at + 30) * k], w, part, k, dxs)
        if at:
            call()
        else:
            kernels |= launched(call, NAMES)
            assert len(kernels) == 4, kernels
        assert torch.equal(ys, y[at * k:(at + 30) * k]) and torch.equal(dxs, dx[at * k:(at + 30) * k])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [8, 24, 32, 40, 64])
@pytest.mark.parametrize("T,N", [(1, 72), (5, 1032), (300, 2056)])
def test_short_sums(T, N, K, dtype):
    """Sums of at most 64: against the formula, and the bits of the kernel for few outputs."""
    k, E = 2, 3
    ids = routing(T, k, E)
    if T > 1:
        ids[T // 2, 0] = -1
    split, _ = make_split(ids, E)
    for by_token, out in ((True, dtype), (False, torch.float32),
                          (True, torch.float16 if dtype == torch.bfloat16 else torch.bfloat16)):
        x, dy, w = inputs(T, k, E, N, K, dtype, by_token, K)
        dev = [v.cuda() for v in (x, dy, w)]
        y, dx, dw = run(*dev, split, k, out, torch.float32)
        check(ids, x, dy, w, y, dx, dw)
        assert launched(lambda: moe.moe_grouped_linear(dev[0], dev[2], split, k, y), NAMES)
        for at in (0, N - 64):
            few = torch.full((T * k, 64), 7.0, dtype=out, device="cuda")
            part = dev[2][:, at:at + 64].contiguous()
            moe.moe_grouped_linear(dev[0], part, split, k, few)
            keep = (ids.reshape(-1) >= 0).cuda()
            assert torch.equal(few[keep], y[keep, at:at + 64])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [8, 16, 24, 32])
@pytest.mark.parametrize("T,K", [(1, 72), (5, 200), (40, 4104), (300, 1000)])
def test_few_outputs(T, N, K, dtype):
    """At most 32 outputs: against the formula, and one token's bits alone and in the step."""
    k, E = 2, 3
    ids = routing(T, k, E)
    if T > 1:
        ids[T // 2, 0] = -1
    split, _ = make_split(ids, E)
    for by_token, out in ((True, dtype), (False, torch.float32),
                          (True, torch.float16 if dtype == torch.bfloat16 else torch.bfloat16)):
        x, dy, w = inputs(T, k, E, N, K, dtype, by_token, K)
        dev = [v.cuda() for v in (x, dy, w)]
        y, dx, dw = run(*dev, split, k, out, torch.float32)
        check(ids, x, dy, w, y, dx, dw)
        got = launched(lambda: moe.moe_grouped_linear(dev[0], dev[2], split, k, y), NAMES)
        assert len(got) == 1 and next(iter(got)).startswith("grouped_narrow<")
        at, per = T - 1, 1 if by_token else k
        alone, _ = make_split(ids[at:], E)
        one = torch.full((k, N), 7.0, dtype=out, device="cuda")
        moe.moe_grouped_linear(dev[0][at * per:(at + 1) * per], dev[2], alone, k, one)
        assert torch.equal(one, y[at * k:])


@pytest.mark.parametrize("T", [500, 521, 2000])
def test_weights_gradient_of_long_groups(T):
    """Groups past the slots that a workgroup holds at once, with rows of other experts
    between theirs, for both kernels."""
    k = 2
    for E, N, K in ((2, 136, 200), (3, 2600, 4616)):
        g = torch.Generator().manual_seed(T)
        ids = (torch.rand(T, k, generator=g) < 0.1).to(torch.int32)
        split, _ = make_split(ids, E)
        x, dy, w = inputs(T, k, E, N, K, torch.bfloat16, T % 2 == 0, T)
        y, dx, dw = run(x.cuda(), dy.cuda(), w.cuda(), split, k, torch.bfloat16, torch.float32)
        check(ids, x, dy, w, y, dx, dw)
