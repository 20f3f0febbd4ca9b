"""Which tiles the products grouped by expert take for narrow results and around one round
of the card, and that the results are the formulas' there."""
import pytest
import torch

import expert_weight_residency_amd as moe
from kernel_instances import launched
from test_gpu_grouped import check, inputs, make_split, routing, run
from test_gpu_grouped_kernels import NAMES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


# T, k, E, N, K, call, start of its kernel's name (bf16): results of at most 128 columns
# never take the tiles of 256, whatever the rows; small tiles while they are about one round
# of two workgroups per CU (256 of them), or for the weights of three.
RULES = [
    (17000, 2, 4, 128, 264, 0, "grouped<0, 0, 128"),
    (17000, 2, 4, 136, 264, 0, "grouped_forward<0>"),
    (17000, 2, 4, 40, 264, 0, "grouped<0, 0, 128"),
    (33000, 2, 4, 264, 128, 1, "grouped<1, 0, 128"),
    (33000, 2, 4, 264, 136, 1, "grouped_gradient<1, 0>"),
    (33000, 2, 4, 264, 16, 1, "grouped<1, 0, 128"),
    (3000, 1, 4, 320, 200, 0, "grouped<0, 0, 64"),
    (3750, 1, 4, 320, 200, 0, "grouped<0, 0, 128"),
    (3000, 1, 4, 200, 320, 1, "grouped<1, 0, 64"),
    (3750, 1, 4, 200, 320, 1, "grouped<1, 0, 128"),
    (200, 1, 3, 1024, 1024, 2, "grouped<2, 0, 64"),
    (200, 1, 4, 1024, 1024, 2, "grouped<2, 0, 128"),
    (200, 1, 5, 1024, 1024, 2, "grouped<2, 0, 64"),
]


@pytest.mark.parametrize("T,k,E,N,K,op,kernel", RULES)
def test_tiles(T, k, E, N, K, op, kernel):
    ids = routing(T, k, E)
    ids[T // 2] = -1
    split, _ = make_split(ids, E)
    x, dy, w = inputs(T, k, E, N, K, torch.bfloat16, False, 7)
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    y, dx, dw = run(xd, dyd, wd, split, k, torch.bfloat16, torch.float32)
    check(ids, x, dy, w, y, dx, dw)
    call = (lambda: moe.moe_grouped_linear(xd, wd, split, k, y), lambda: moe.moe_grouped_linear_dx(dyd, wd, split, k, dx),
            lambda: moe.moe_grouped_linear_dw(dyd, xd, split, k, dw))[op]
    got = launched(call, NAMES)
    assert len(got) == 1 and next(iter(got)).startswith(kernel), got
