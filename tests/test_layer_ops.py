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
    def call(logits=P, dtype=2, ld=384, T=4, E=384, k=6, norm=0, ids=4 * P, w=8 * P):
        return L.moe_topk_gate(logits, dtype, ld, T, E, k, norm, ids, w, None)
    for kw, text in (({"dtype": 3}, "dtype"), ({"dtype": -1}, "dtype"), ({"norm": 2}, "norm"),
                     ({"T": -1}, "T="), ({"E": 0, "ld": 0}, "E="), ({"E": 4097, "ld": 5000}, "E="),
                     ({"k": 0}, "k="), ({"k": 33}, "k="), ({"E": 4, "k": 5}, "k="),
                     ({"ld": 383}, "ld="), ({"ld": 2 ** 32}, "ld="), ({"T": 2 ** 25 + 1}, "T="),
                     ({"logits": None}, "NULL"), ({"ids": None}, "NULL"), ({"w": None}, "NULL"),
                     ({"logits": P + 2}, "aligned"), ({"ids": P + 2}, "aligned"),
                     ({"ids": P + 64}, "overlap"), ({"w": P + 6100}, "overlap"),
                     ({"w": 4 * P + 92}, "overlap"),
                     ({"logits": P + 1, "dtype": 0}, "aligned")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    assert call(T=0, logits=None, ids=None, w=None) == moe.MOE_OK
    assert moe.moe_last_error() == ""


def test_few_refusals(L):
    def bank(p=P, n=4, on=0):
        return moe.MoeBankC(p, p, p, p, n, on)

    def call(hot=None, cold=None, rm=P, E=8, x=P, ids=P, w=P, T=4, k=2, H=256, I=128, ninv=P,
             ws=8 * P, out=2 * P, null=False):
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
                     ({"ws": P}, "overlap"), ({"ws": 2 * P - 64}, "overlap"),
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


def test_quantize_refusals(L):
    def call(x=P, dtype=0, ld=64, rows=4, K=64, q=8 * P, s=4 * P):
        return L.moe_quantize_rows_i8(x, dtype, ld, rows, K, q, s, None)
    for kw, text in (({"dtype": 9}, "dtype"), ({"rows": -1}, "rows"), ({"rows": 2 ** 23 + 1}, "rows"), ({"K": 0, "ld": 0}, "K="),
                     ({"K": 131073, "ld": 131073}, "K="), ({"ld": 63}, "ld="),
                     ({"x": None}, "NULL"), ({"q": None}, "NULL"), ({"s": None}, "NULL"),
                     ({"x": P + 1}, "aligned"), ({"s": P + 2}, "aligned"),
                     ({"q": P + 100}, "overlap"), ({"s": P + 8}, "overlap"),
                     ({"s": 8 * P + 16}, "overlap")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    assert call(rows=0, x=None) == moe.MOE_OK


def test_linear_refusals(L):
    def call(xq=P, ldx=64, xs=P, M=4, w=2 * P, ws=P, N=8, K=64, y=8 * P, dtype=0, ldy=8):
        return L.moe_linear_i8(xq, ldx, xs, M, w, ws, N, K, y, dtype, ldy, None)
    for kw, text in (({"dtype": 3}, "dtype"), ({"M": -1}, "M="), ({"N": -1}, "N="),
                     ({"M": 2 ** 23 + 1}, "M="), ({"N": 2 ** 23 + 1, "ldy": 2 ** 24}, "N="),
                     ({"K": 0}, "K="), ({"K": 24}, "K="), ({"K": 131088, "ldx": 131088}, "K="),
                     ({"ldx": 48}, "ldx"), ({"ldx": 72}, "ldx"), ({"ldy": 7}, "ldy"),
                     ({"xq": None}, "NULL"), ({"xs": None}, "NULL"), ({"w": None}, "NULL"),
                     ({"ws": None}, "NULL"), ({"y": None}, "NULL"), ({"xq": P + 8}, "aligned"),
                     ({"w": P + 4}, "aligned"), ({"y": 8 * P + 1}, "aligned"),
                     ({"xs": P + 1}, "aligned"), ({"y": P + 16}, "overlap"),
                     ({"y": 2 * P + 32}, "overlap")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    refused(call(M=2 ** 21, N=2 ** 21, ldy=2 ** 21, K=16, xq=2 ** 44, w=2 ** 45, y=2 ** 50),
            moe.MOE_ENOTSUP, "tiles")
    assert call(M=0, xq=None) == moe.MOE_OK and call(N=0, ldy=0, w=None) == moe.MOE_OK


def test_ffn_i8_refusals(L):
    def call(bank=None, split=P, xq=P, xs=P, T=4, k=2, H=256, I=128, ws=P, Y=P):
        bank = moe.MoeBankC(P, P, P, P, 4, 0) if bank is None else bank
        sp = moe.MoeSplitC(split, split, split, split)
        return L.moe_expert_ffn_i8(ctypes.byref(bank) if bank else None, sp, xq, xs, T, k, H, I, ws,
                                   Y, None)
    for kw, text in (({"T": -1}, "T="), ({"k": 0}, "k="), ({"k": 33}, "k="),
                     ({"T": 2 ** 22 + 1}, "T*k"), ({"H": 100}, "multiples"), ({"I": 0}, "multiples"),
                     ({"bank": 0}, "NULL"), ({"bank": moe.MoeBankC(P, P, P, P, 5000, 0)}, "rows"),
                     ({"split": 0}, "split"), ({"xq": None}, "NULL"), ({"xs": None}, "NULL"),
                     ({"ws": None}, "NULL"), ({"Y": None}, "NULL"), ({"xq": P + 8}, "aligned"),
                     ({"Y": P + 2}, "aligned"), ({"ws": P + 4}, "aligned"),
                     ({"bank": moe.MoeBankC(P, P + 4, P, P, 4, 0)}, "aligned"),
                     ({"bank": moe.MoeBankC(P, P, P, P, 4, 7)}, "on_host")):
        refused(call(**kw), moe.MOE_EINVAL, text)
    refused(call(H=32832), moe.MOE_ENOTSUP, "supported")
    refused(call(T=2 ** 22, H=32768, I=32768), moe.MOE_ENOTSUP, "tiles")
    assert call(T=0, xq=None) == moe.MOE_OK
    assert call(bank=moe.MoeBankC(0, 0, 0, 0, 0, 0)) == moe.MOE_OK
    assert moe.moe_ffn_i8_workspace_bytes(16, 6, 4096, 2880) == 96 * (2880 * 5 + 4)
    assert moe.moe_ffn_i8_workspace_bytes(16, 0, 4096, 2880) == 0


def test_residency_layer_refuses_mixed_and_staged_i8():
    from expert_weight_residency_amd.layer import ResidencyLayer
    z = torch.zeros(1, 64, 64, dtype=torch.int8)
    s = torch.zeros(1, 64)
    i8 = moe.BankI8(z, s, z, s)
    u = torch.zeros(1, 64, 64, dtype=torch.uint8)
    fp4 = moe.Bank(u, u, u, u)
    rm = torch.zeros(2, dtype=torch.int32)
    for hot, cold, stage in ((i8, fp4, None), (fp4, i8, None), (i8, i8, object())):
        with pytest.raises(moe.MoeError) as e:
            ResidencyLayer(hot, cold, rm, 64, 64, stage=stage)
        assert e.value.code == moe.MOE_EINVAL
    layer = ResidencyLayer(fp4, fp4, rm, 64, 64)
    with pytest.raises(moe.MoeError):
        layer.route(torch.zeros(1, 3), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1))


def test_tensors_on_another_device_are_refused():
    class On:  # what the check looks at of a tensor
        def __init__(self, dev):
            self.dev = dev
        is_cuda = True
        device = "cuda:1"

        def get_device(self):
            return self.dev
    moe._on(0, a=On(0), b=None, c=torch.zeros(1))
    with pytest.raises(moe.MoeError) as e:
        moe._on(0, a=On(0), b=On(1))
    assert e.value.code == moe.MOE_EINVAL and "b: on cuda:1" in str(e.value)


def test_streams_of_another_device_are_refused(monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(moe.MoeError) as e:
        moe._current(Stream())
    assert e.value.code == moe.MOE_EINVAL and "stream" in str(e.value)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert moe._current(Stream())[0] == 1
    assert moe._current(77) == (1, 77)  # a raw handle


@pytest.mark.parametrize("T", [1, 16, 17, 40, 300])
def test_buffers_serve_few_token_steps_of_any_size(T):
    from expert_weight_residency_amd.layer import LayerBuffers
    k, H, I = 2, 256, 64  # tables larger than a token's h rows
    bufs = LayerBuffers.allocate(T, k, H, I, 4, 4, device="cpu")
    for t in range(1, min(T, 16) + 1):
        assert bufs.workspace.numel() >= moe.moe_layer_few_workspace_bytes(t, k, H, I)


class Recorder:
    """Stands in for the streams and the entry points that ResidencyLayer calls:
    every operation knows which others it waits for."""

    def __init__(self, monkeypatch):
        from expert_weight_residency_amd import layer
        self.after = {}  # operation -> those it follows, directly or not
        self.args = {}
        for name in ("moe_route_split", "moe_quantize_rows_i8", "moe_expert_ffn_i8",
                     "moe_expert_ffn_mxfp4", "moe_finalize"):
            monkeypatch.setattr(layer, name, lambda *a, _name=name, stream=None, **kw:
                                self.call(_name, a, stream))

    def call(self, name, args, stream):
        if name.startswith("moe_expert_ffn"):
            name = args[0].name
        self.after[name], self.args[name] = set(stream.done), args
        stream.done.add(name)

    class Stream:
        def __init__(self):
            self.done = set()

        def wait_stream(self, other):
            self.done |= other.done


def stub_i8_layer(T, H, I, x_dtype=torch.bfloat16):
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer

    def bank(name):
        b = moe.BankI8(torch.zeros(1, 2 * I, H, dtype=torch.int8), torch.zeros(1, 2 * I),
                       torch.zeros(1, H, I, dtype=torch.int8), torch.zeros(1, H))
        b.name = name
        return b
    layer = ResidencyLayer(bank("hot"), bank("cold"), torch.tensor([0, -1], dtype=torch.int32), H, I)
    bufs = LayerBuffers.allocate(T, 1, H, I, 1, 1, device="cpu", i8=True)
    x = torch.zeros(T, H, dtype=torch.int16).view(x_dtype)
    return layer, bufs, (x, torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1))


@pytest.mark.parametrize("side", [(), ("cold_stream",), ("hot_stream",), ("hot_stream", "cold_stream")])
def test_i8_banks_run_beside_each_other(monkeypatch, side):
    """With a side stream neither bank's FFN waits for the other's; both follow
    the split and the quantisation, and the finalize follows both."""
    rec = Recorder(monkeypatch)
    layer, bufs, args = stub_i8_layer(2, 64, 64)
    s, other = Recorder.Stream(), {n: Recorder.Stream() for n in side}
    layer.forward(*args, bufs, stream=s, **other)
    first = {"moe_route_split", "moe_quantize_rows_i8"}
    assert first <= rec.after["hot"] and first <= rec.after["cold"]
    assert {"hot", "cold"} <= rec.after["moe_finalize"]
    if side:
        assert "cold" not in rec.after["hot"] and "hot" not in rec.after["cold"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int16, torch.uint16])
def test_i8_banks_take_bf16_bits_in_any_type(monkeypatch, dtype):
    rec = Recorder(monkeypatch)
    layer, bufs, args = stub_i8_layer(2, 64, 64, dtype)
    layer.forward(*args, bufs, stream=Recorder.Stream())
    x = rec.args["moe_quantize_rows_i8"][0]
    assert x.dtype == torch.bfloat16 and x.data_ptr() == args[0].data_ptr()


def test_ffn_i8_refuses_overlapping_buffers(L):
    T, k, H, I = 4, 2, 256, 128
    n = {"xq": T * H, "xs": 4 * T, "ws": moe.moe_ffn_i8_workspace_bytes(T, k, H, I), "Y": 2 * T * k * H}
    bank, split = moe.MoeBankC(P, P, P, P, 4, 0), moe.MoeSplitC(P, P, P, P)
    for a, b in (("Y", "ws"), ("Y", "xq"), ("Y", "xs"), ("ws", "xq"), ("ws", "xs")):
        at = {"xq": 2 * P, "xs": 4 * P, "ws": 8 * P, "Y": 16 * P}
        for shift in (0, n[b] - 16, -(n[a] - 16)):  # the same place, the last and first bytes shared
            at[a] = at[b] + shift // 16 * 16
            rc = L.moe_expert_ffn_i8(ctypes.byref(bank), split, at["xq"], at["xs"], T, k, H, I, at["ws"],
                                     at["Y"], None)
            refused(rc, moe.MOE_EINVAL, "overlap")


def test_few_refuses_misaligned_and_overlapping_arrays(L):
    T, k, E, H, I = 4, 2, 8, 256, 128
    n = {"rm": 4 * E, "ids": 4 * T * k, "w": 4 * T * k, "x": 2 * T * H, "ninv": 4, "counts": 4 * E,
         "ws": moe.moe_layer_few_workspace_bytes(T, k, H, I), "out": 2 * T * H}
    bank = moe.MoeBankC(P, P, P, P, 4, 0)

    def call(**move):
        at = {**{name: (2 + 2 * i) * P for i, name in enumerate(n)}, **move}
        return L.moe_layer_few_mxfp4(ctypes.byref(bank), ctypes.byref(bank), at["rm"], E, at["x"], at["ids"],
                                     at["w"], T, k, H, I, at["counts"], 256, at["ninv"], at["ws"], at["out"],
                                     None)
    for name in ("rm", "ids", "w", "ninv", "counts"):
        refused(call(**{name: 64 * P + 2}), moe.MOE_EINVAL, "aligned")
    for a in ("ninv", "counts", "ws", "out"):
        for b in n:
            if a != b:
                for at in (64 * P, 64 * P + (n[b] - 1) // 16 * 16, 64 * P - (n[a] - 1) // 16 * 16):
                    refused(call(**{a: at, b: 64 * P}), moe.MOE_EINVAL, "overlap")
