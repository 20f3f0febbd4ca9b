"""What the 8-bit floating point products refuse, without a GPU: every check of the
C ABI and of the binding runs before any GPU call."""
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


def test_quantize_refusals(L):
    def call(x=P, dtype=0, ld=64, rows=4, K=64, q=8 * P, s=4 * P):
        return L.moe_quantize_rows_f8(x, dtype, ld, rows, K, q, s, None)
    for kw, text in (({"dtype": 9}, "dtype"), ({"rows": -1}, "rows"), ({"rows": 2 ** 23 + 1}, "rows"),
                     ({"K": 0, "ld": 0}, "K="), ({"K": 131073, "ld": 131073}, "K="), ({"ld": 63}, "ld="),
                     ({"ld": 2 ** 31 + 1}, "ld="), ({"x": None}, "NULL"), ({"q": None}, "NULL"),
                     ({"s": None}, "NULL"), ({"x": P + 1}, "aligned"), ({"s": P + 2}, "aligned"),
                     ({"x": P + 2, "dtype": 2}, "aligned"), ({"q": P + 100}, "overlap"),
                     ({"s": P + 8}, "overlap"), ({"s": 8 * P + 16}, "overlap"), ({"s": 8 * P - 12}, "overlap"),
                     # two blocks a row: 8 bytes of scales each
                     ({"s": 8 * P - 28, "K": 129, "ld": 129}, "overlap")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    assert call(rows=0, x=None) == moe.MOE_OK


def test_linear_refusals(L):
    def call(xq=P, ldx=64, xs=P, M=4, w=2 * P, ws=P, N=8, K=64, y=8 * P, dtype=0, ldy=8):
        return L.moe_linear_f8(xq, ldx, xs, M, w, ws, N, K, y, dtype, ldy, None)
    for kw, text in (({"dtype": 3}, "dtype"), ({"M": -1}, "M="), ({"N": -1}, "N="),
                     ({"M": 2 ** 23 + 1}, "M="), ({"N": 2 ** 23 + 1, "ldy": 2 ** 24}, "N="),
                     ({"K": 0}, "K="), ({"K": 24}, "K="), ({"K": 131088, "ldx": 131088}, "K="),
                     ({"ldx": 48}, "ldx"), ({"ldx": 72}, "ldx"), ({"ldy": 7}, "ldy"),
                     ({"xq": None}, "NULL"), ({"xs": None}, "NULL"), ({"w": None}, "NULL"),
                     ({"ws": None}, "NULL"), ({"y": None}, "NULL"), ({"xq": P + 8}, "aligned"),
                     ({"w": P + 4}, "aligned"), ({"y": 8 * P + 1}, "aligned"), ({"xs": P + 1}, "aligned"),
                     ({"ws": P + 2}, "aligned"), ({"y": P + 16}, "overlap"), ({"y": 2 * P + 32}, "overlap"),
                     ({"xs": 8 * P + 48}, "overlap"), ({"ws": 8 * P + 60}, "overlap"),
                     ({"xs": 8 * P - 12}, "overlap")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    refused(call(M=2 ** 21, N=2 ** 21, ldy=2 ** 21, K=16, xq=2 ** 44, w=2 ** 45, y=2 ** 50),
            moe.MOE_ENOTSUP, "tiles")
    assert call(M=0, xq=None) == moe.MOE_OK and call(N=0, ldy=0, w=None) == moe.MOE_OK


def test_ffn_refusals(L):
    def call(bank=None, split=P, xq=P, xs=P, T=4, k=2, H=256, I=128, ws=P, Y=P):
        bank = moe.MoeBankC(P, P, P, P, 4, 0) if bank is None else bank
        sp = moe.MoeSplitC(split, split, split, split)
        return L.moe_expert_ffn_f8(ctypes.byref(bank) if bank else None, sp, xq, xs, T, k, H, I, ws,
                                   Y, None)
    for kw, text in (({"T": -1}, "T="), ({"k": 0}, "k="), ({"k": 33}, "k="),
                     ({"T": 2 ** 22 + 1}, "T*k"), ({"H": 100}, "multiples"), ({"I": 0}, "multiples"),
                     ({"bank": 0}, "NULL"), ({"bank": moe.MoeBankC(P, P, P, P, 5000, 0)}, "rows"),
                     ({"split": 0}, "split"), ({"xq": None}, "NULL"), ({"xs": None}, "NULL"),
                     ({"ws": None}, "NULL"), ({"Y": None}, "NULL"), ({"xq": P + 8}, "aligned"),
                     ({"Y": P + 2}, "aligned"), ({"ws": P + 4}, "aligned"), ({"xs": P + 2}, "aligned"),
                     ({"bank": moe.MoeBankC(P, P + 4, P, P, 4, 0)}, "aligned"),
                     ({"bank": moe.MoeBankC(P, P, P, P, 4, 7)}, "on_host")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    refused(call(H=32832), moe.MOE_ENOTSUP, "supported")
    refused(call(T=2 ** 22, H=32768, I=32768), moe.MOE_ENOTSUP, "tiles")
    assert call(T=0, xq=None) == moe.MOE_OK
    assert call(bank=moe.MoeBankC(0, 0, 0, 0, 0, 0)) == moe.MOE_OK
    assert moe.moe_ffn_f8_workspace_bytes(16, 0, 4096, 2880) == 0
    assert moe.moe_ffn_f8_workspace_bytes(16, 6, 4096, 2880) > 96 * 2880


def test_ffn_refuses_overlapping_buffers(L):
    T, k, H, I = 4, 2, 256, 128
    n = {"xq": T * H, "xs": 8 * T, "ws": moe.moe_ffn_f8_workspace_bytes(T, k, H, I), "Y": 2 * T * k * H}
    bank, split = moe.MoeBankC(P, P, P, P, 4, 0), moe.MoeSplitC(P, P, P, P)
    for a, b in (("Y", "ws"), ("Y", "xq"), ("Y", "xs"), ("ws", "xq"), ("ws", "xs")):
        at = {"xq": 2 * P, "xs": 4 * P, "ws": 8 * P, "Y": 16 * P}
        for shift in (0, n[b] - 16, -(n[a] - 16)):  # the same place, the last and first bytes shared
            at[a] = at[b] + shift // 16 * 16
            rc = L.moe_expert_ffn_f8(ctypes.byref(bank), split, at["xq"], at["xs"], T, k, H, I, at["ws"],
                                     at["Y"], None)
            refused(rc, moe.MOE_EINVAL, "overlap")


def test_binding_refuses_host_tensors_and_wrong_types():
    f8 = torch.float8_e4m3fn
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 64).to(f8), torch.zeros(2, 1)
    for call in (lambda: moe.moe_quantize_rows_f8(x, q, s),
                 lambda: moe.moe_linear_f8(q, s, q, s[:1], torch.zeros(2, 2)),
                 lambda: moe.moe_linear_f8(x, s, q, s[:1], torch.zeros(2, 2)),
                 lambda: moe.BankF8(x, s, q, s).abi(),
                 lambda: moe.BankF8(q.view(1, 2, 64), s, q.view(1, 2, 64), s, 5).abi()):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_EINVAL


def test_residency_layer_refuses_mixed_banks_and_buffers():
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    z = torch.zeros(1, 64, 64)
    s = torch.zeros(1, 64)
    i8 = moe.BankI8(z.to(torch.int8), s, z.to(torch.int8), s)
    f8 = moe.BankF8(z.to(torch.float8_e4m3fn), s, z.to(torch.float8_e4m3fn), s)
    u = z.to(torch.uint8)
    fp4 = moe.Bank(u, u, u, u)
    rm = torch.zeros(2, dtype=torch.int32)
    for hot, cold, stage in ((f8, fp4, None), (fp4, f8, None), (i8, f8, None), (f8, i8, None),
                             (f8, f8, object())):
        with pytest.raises(moe.MoeError) as e:
            ResidencyLayer(hot, cold, rm, 64, 64, stage=stage)
        assert e.value.code == moe.MOE_EINVAL
    with pytest.raises(moe.MoeError):
        LayerBuffers.allocate(2, 1, 64, 64, 1, 1, device="cpu", i8=True, f8=True)
