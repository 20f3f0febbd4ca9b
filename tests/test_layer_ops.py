"""What the operators around the residency split refuse, without a GPU: every
check of the C ABI and of the binding runs before any GPU call."""
import ctypes

import pytest
import torch

import expert_weight_residency_amd as moe

P = 0x10000  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def refused(rc, code, text):
    assert rc == code and text in moe.moe_last_error(), (rc, moe.moe_last_error())


def test_gate_refusals(L):
    def call(logits=P, dtype=2, ld=384, T=4, E=384, k=6, norm=0, ids=P, w=P):
        return L.moe_topk_gate(logits, dtype, ld, T, E, k, norm, ids, w, None)
    for kw, text in (({"dtype": 3}, "dtype"), ({"dtype": -1}, "dtype"), ({"norm": 2}, "norm"),
                     ({"T": -1}, "T="), ({"E": 0, "ld": 0}, "E="), ({"E": 4097, "ld": 5000}, "E="),
                     ({"k": 0}, "k="), ({"k": 33}, "k="), ({"E": 4, "k": 5}, "k="),
                     ({"ld": 383}, "ld="), ({"ld": 2 ** 32}, "ld="), ({"T": 2 ** 30}, "T*k"),
                     ({"logits": None}, "NULL"), ({"ids": None}, "NULL"), ({"w": None}, "NULL"),
                     ({"logits": P + 2}, "aligned"), ({"ids": P + 2}, "aligned"),
                     ({"logits": P + 1, "dtype": 0}, "aligned")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    assert call(T=0, logits=None, ids=None, w=None) == moe.MOE_OK
    assert moe.moe_last_error() == ""


def test_few_refusals(L):
    def bank(p=P, n=4, on=0):
        return moe.MoeBankC(p, p, p, p, n, on)

    def call(hot=None, cold=None, rm=P, E=8, x=P, ids=P, w=P, T=4, k=2, H=256, I=128, ninv=P,
             ws=P, out=2 * P, null=False):
        hot, cold = hot or bank(), cold or bank()
        h = None if null else ctypes.byref(hot)
        return L.moe_layer_few_mxfp4(h, ctypes.byref(cold), rm, E, x, ids, w, T, k, H, I, None,
                                     256, ninv, ws, out, None)
    for kw, text in (({"T": -1}, "T="), ({"k": 0}, "k="), ({"k": 33}, "k="), ({"E": 0}, "E="),
                     ({"E": 4097}, "E="), ({"H": 100}, "multiples"), ({"I": 0}, "multiples"),
                     ({"null": True}, "NULL"), ({"hot": bank(n=-1)}, "rows"),
                     ({"cold": bank(n=4097)}, "rows"), ({"rm": None}, "NULL"),
                     ({"x": None}, "NULL"), ({"ids": None}, "NULL"), ({"w": None}, "NULL"),
                     ({"ninv": None}, "NULL"), ({"ws": None}, "NULL"), ({"out": None}, "NULL"),
                     ({"x": P + 8}, "aligned"), ({"ws": P + 8}, "aligned"),
                     ({"out": P}, "overlap"), ({"out": P + 4 * 256 * 2 - 16}, "overlap"),
                     ({"hot": bank(on=3)}, "on_host"), ({"hot": bank(p=0)}, "NULL"),
                     ({"cold": bank(p=P + 8)}, "aligned")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    for kw in ({"T": 17}, {"H": 8256}, {"I": 4160}):
        refused(call(**kw), moe.MOE_ENOTSUP, "supported")
        T, H, I = kw.get("T", 4), kw.get("H", 256), kw.get("I", 128)
        assert moe.moe_layer_few_workspace_bytes(T, 2, H, I) == 0
    assert call(T=0, x=None, ids=None, w=None, out=None) == moe.MOE_OK
    assert moe.moe_layer_few_workspace_bytes(16, 6, 4096, 2880) >= 16 * 6 * 2880 * 2
    assert moe.moe_layer_few_workspace_bytes(0, 6, 4096, 2880) == 0


def test_binding_refuses_host_and_odd_tensors():
    l = torch.zeros(4, 8)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_topk_gate(l, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    assert e.value.code == moe.MOE_EINVAL
    with pytest.raises(moe.MoeError):
        moe.moe_topk_gate(l.to(torch.int32), torch.zeros(4, 2, dtype=torch.int32),
                          torch.zeros(4, 2))
