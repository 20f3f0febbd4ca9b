"""What the products grouped by expert refuse, without a GPU: every check of the C ABI
and of the binding runs before any GPU call."""
import pytest
import torch

import expert_weight_residency_amd as moe

P = 0x100000  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def refused(rc, code, text):
    assert rc == code and text in moe.moe_last_error(), (rc, moe.moe_last_error())


def calls(L):
    """The three calls with the same names of arguments: a and b the inputs, o the output."""
    def split(p):
        return moe.MoeSplitC(p, p, p, p)

    def forward(a=P, b=2 * P, o=4 * P, dt=0, ot=0, bt=1, rows=4, host=0, sp=P, T=4, k=2, N=64, K=128):
        return L.moe_grouped_linear(a, dt, bt, b, rows, host, split(sp), T, k, N, K, o, ot, None)

    def dx(a=P, b=2 * P, o=4 * P, dt=0, ot=0, bt=1, rows=4, host=0, sp=P, T=4, k=2, N=64, K=128):
        return L.moe_grouped_linear_dx(a, dt, b, rows, host, split(sp), T, k, N, K, o, ot, None)

    def dw(a=P, b=2 * P, o=4 * P, dt=0, ot=0, bt=1, rows=4, host=0, sp=P, T=4, k=2, N=64, K=128):
        return L.moe_grouped_linear_dw(a, b, dt, bt, rows, split(sp), T, k, N, K, o, ot, None)
    return forward, dx, dw


@pytest.mark.parametrize("which", [0, 1, 2])
def test_refusals(L, which):
    call = calls(L)[which]
    for kw, text in (({"dt": 2}, "dtype"), ({"dt": -1}, "dtype"), ({"ot": 3}, "dtype"), ({"T": -1}, "T="),
                     ({"k": 0}, "k="), ({"k": 33}, "k="), ({"T": 2 ** 22 + 1}, "T*k"),
                     ({"rows": -1}, "rows"), ({"rows": 4097}, "rows"), ({"N": 0}, "N="), ({"N": 12}, "N="),
                     ({"K": 4}, "K="), ({"K": 131080}, "K="), ({"N": 131080}, "N="),
                     ({"sp": 0}, "split"), ({"a": None}, "NULL"), ({"b": None}, "NULL"), ({"o": None}, "NULL"),
                     ({"a": P + 8}, "aligned"), ({"b": P + 2}, "aligned"), ({"o": P + 4}, "aligned"),
                     ({"o": P}, "overlap"), ({"o": 2 * P}, "overlap"), ({"o": P + 4 * 64 * 2 - 16}, "overlap"),
                     ({"o": 2 * P + 16}, "overlap")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    if which < 2:
        refused(call(host=2), moe.MOE_EINVAL, "on_host")
        assert call(T=0, a=None, o=None) == moe.MOE_OK
    assert call(rows=0, a=None, b=None, o=None) == moe.MOE_OK
    assert moe.moe_last_error() == ""


def test_too_many_tiles(L):
    forward, dx, dw = calls(L)
    far = {"a": 2 ** 44, "b": 2 ** 50, "o": 2 ** 54}
    refused(forward(T=2 ** 22, N=131072, K=64, **far), moe.MOE_ENOTSUP, "tiles")
    refused(dx(T=2 ** 22, N=64, K=131072, **far), moe.MOE_ENOTSUP, "tiles")
    refused(dw(rows=4096, N=8192, K=8192, **far), moe.MOE_ENOTSUP, "tiles")


def test_outputs_last_bytes_count(L):
    """Each input's last 16 bytes and the output's, of every type and row form."""
    forward, dx, dw = calls(L)
    T, k, N, K, R = 4, 2, 64, 128, 4
    for ot, size in ((0, 2), (1, 2), (2, 4)):
        for call, bt, a, b, o in ((forward, 1, T * K * 2, R * N * K * 2, T * k * N * size),
                                  (forward, 0, T * k * K * 2, R * N * K * 2, T * k * N * size),
                                  (dx, 0, T * k * N * 2, R * N * K * 2, T * k * K * size),
                                  (dw, 1, T * k * N * 2, T * K * 2, R * N * K * size),
                                  (dw, 0, T * k * N * 2, T * k * K * 2, R * N * K * size)):
            at = {"bt": bt, "ot": ot}
            refused(call(o=P + a - 16, **at), moe.MOE_EINVAL, "overlap")
            refused(call(o=P - o + 16, **at), moe.MOE_EINVAL, "overlap")
            refused(call(o=8 * P + b - 16, b=8 * P, **at), moe.MOE_EINVAL, "overlap")
            refused(call(o=8 * P - o + 16, b=8 * P, **at), moe.MOE_EINVAL, "overlap")


def test_binding_refuses_host_tensors():
    sp = moe.Split.empty(2, 2, 2, device="cpu")
    x, w, y = torch.zeros(2, 8).bfloat16(), torch.zeros(2, 8, 8).bfloat16(), torch.zeros(4, 8).bfloat16()
    moe_calls = (lambda: moe.moe_grouped_linear(x, w, sp, 2, y),
                 lambda: moe.moe_grouped_linear_dx(y, w, sp, 2, y.clone()),
                 lambda: moe.moe_grouped_linear_dw(y, x, sp, 2, w))
    for call in moe_calls:
        with pytest.raises((moe.MoeError, RuntimeError)):
            call()


@pytest.mark.parametrize("rows,k,ok", [(4, 2, True), (5, 2, False), (0, 3, True), (4, 0, False), (6, 2, False)])
def test_binding_checks_the_slots(rows, k, ok):
    sp = moe.Split.empty(2, 2, 2, device="cpu")  # 4 slots
    if ok:
        assert moe._grouped_split(sp, rows, k) == rows // k
    else:
        with pytest.raises(moe.MoeError):
            moe._grouped_split(sp, rows, k)


@pytest.mark.parametrize("made_for", [(2, 4, 2), (8, 2, 2)])
def test_binding_checks_the_splits_capacity(made_for):
    """A split of fewer experts or a shorter step: the kernels would read past its end."""
    n_rows, T, k = 8, 4, 2
    with pytest.raises(moe.MoeError, match="split"):
        moe._grouped_split(moe.Split.empty(*made_for, device="cpu"), T * k, k, n_rows)
    assert moe._grouped_split(moe.Split.empty(n_rows, T, k, device="cpu"), T * k, k, n_rows) == T
    # a larger one serves a shorter step and fewer rows
    assert moe._grouped_split(moe.Split.empty(n_rows, T, k, device="cpu"), 2 * k, k, 2) == 2


def test_binding_tells_rows_of_tokens_from_rows_of_slots():
    assert moe._grouped_by_token(torch.zeros(3, 8), 3, 2) == 1
    assert moe._grouped_by_token(torch.zeros(6, 8), 3, 2) == 0
    assert moe._grouped_by_token(torch.zeros(3, 8), 3, 1) == 1  # one and the same
    for bad in (torch.zeros(5, 8), torch.zeros(3, 8, 1)):
        with pytest.raises(moe.MoeError):
            moe._grouped_by_token(bad, 3, 2)
