"""The 8-bit integer products against their 64-bit forms: the quantised rows
exactly, the dense product within its three fp32 roundings and the output's,
the expert FFN within what the fp32 errors of h can turn in its quantisation;
strides, odd sizes, both kernel families, banks, streams and HIP graphs."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import layer_ref
import synth
from layer_ref import HALF_STEP, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def quantize(x, stream=None):
    rows, K = x.shape
    q = torch.full((rows + 1, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), 99.0, device="cuda")
    torch.cuda.synchronize()
    moe.moe_quantize_rows_i8(x, q[:rows], s[:rows], stream=stream)
    torch.cuda.synchronize()
    assert (q[rows] == 99).all() and s[rows] == 99.0
    return q[:rows], s[:rows]


def check_quantize(x):
    q, s = quantize(x)
    rq, _ = layer_ref.quantize(x.cpu())
    most = x.cpu().float().abs().amax(dim=1)
    assert torch.equal(q.cpu().double(), rq)
    # one fp32 division, rounded to nearest by both
    assert np.array_equal(s.cpu().numpy(), most.numpy() / np.float32(127))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 8), (2, 16), (9, 100), (4, 512), (3, 520),
                                    (2, 2048), (7, 4096), (1, 4104), (2, 8192), (2, 8200),
                                    (1, 32768), (70, 2880)])
def test_quantize_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * 131 + K)
    x = (torch.randn(rows, K, generator=g) * torch.logspace(-3, 3, rows)[:, None]).to(dtype)
    check_quantize(x.cuda())


def test_quantize_ties_and_signs():
    # max 254: every odd integer is a tie; max 127 and halves: likewise
    t = torch.arange(-254, 255, dtype=torch.float32)
    x = torch.stack([t, t / 2, t * 2.0 ** -60, t * 2.0 ** 60])
    for dtype in (torch.float32, torch.bfloat16):
        check_quantize(x.to(dtype).cuda())
    # ties of a maximum that is no power of two times 127: 127 x / m = n + 1/2 exactly
    m = 127.0 * 3
    y = torch.tensor([[m] + [1.5 * (2 * n + 1) for n in range(127)]])
    check_quantize(y.cuda())
    q, _ = quantize(y.cuda())
    assert q[0, 1:5].tolist() == [0, 2, 2, 4]
    # values one fp32 step beside a tie
    z = torch.tensor([1.5 * (2 * n + 1) for n in range(127)])
    up, dn = torch.nextafter(z, torch.tensor(1e9)), torch.nextafter(z, torch.tensor(0.0))
    check_quantize(torch.cat([torch.tensor([m]), up, dn]).view(1, -1).cuda())


def test_quantize_strides_and_offsets():
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(6, 203, generator=g).cuda()
    check_quantize(wide[:, 1:98])          # rows 4 bytes off a 16-byte boundary
    check_quantize(wide.half()[:, :200])   # vectors' length, unaligned row stride
    check_quantize(wide[::2, :100])
    flat = torch.zeros(2 * 2 ** 30 + 64, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((3, 64), (2 ** 30, 1))  # the third row 4 GB on
    far.copy_(torch.randn(3, 64, generator=g).to(torch.bfloat16))
    check_quantize(far)


def test_quantize_special_rows():
    x = torch.randn(7, 64, generator=torch.Generator().manual_seed(6))
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 63] = float("nan")
    x[3] *= 1e-40                     # the scale would be subnormal
    x[4, 0] = torch.finfo(torch.float32).max
    x[5] = -0.0
    q, s = quantize(x.cuda())
    assert (q[[0, 1, 2, 3, 5]] == 0).all()
    assert s[0] == 0 and s[3] == 0 and s[5] == 0 and s[1].isnan() and s[2].isnan()
    check_quantize(x[[4, 6]].cuda())
    y = torch.empty(7, 8, device="cuda")
    w = torch.ones(8, 64, dtype=torch.int8, device="cuda")
    moe.moe_linear_i8(q, s, w, torch.ones(8, device="cuda"), y)
    torch.cuda.synchronize()
    assert y[[1, 2]].isnan().all() and (y[[0, 3, 5]] == 0).all() and y[6].isfinite().all()


def make_linear(M, N, K, seed, extreme=False):
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, generator=g)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, generator=g)
    if extreme:
        xq[0], w[0] = 127, -128   # the largest sums there are
    xs = torch.rand(M, generator=g) + 0.01
    ws = torch.rand(N, generator=g) / (73 * K ** 0.5)
    return xq, xs, w, ws


def check_linear(y, xq, xs, w, ws):
    ref = (xq.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    # the sum to fp32, two products, the type's rounding (and fp16's subnormals)
    tol = (3.1 * U32 + HALF_STEP[y.dtype]) * ref.abs() + (2.0 ** -25 if y.dtype == torch.float16
                                                         else 2.0 ** -140)
    off = (y.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


LINEAR = [(1, 1, 16), (1, 7, 32), (1, 5760, 4096), (3, 100, 2880), (8, 64, 1024), (9, 63, 1040),
          (16, 333, 4096), (16, 40, 8192), (2, 24, 8208), (17, 65, 128), (64, 64, 64),
          (100, 130, 272), (257, 511, 1040), (33, 4096, 2880), (1001, 2047, 1040),
          (4095, 4100, 144), (300, 257, 16), (5, 3, 131056)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K):
    xq, xs, w, ws = make_linear(M, N, K, M + N + K, extreme=True)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        moe.moe_linear_i8(xq.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y[:M])
        torch.cuda.synchronize()
        assert (y[M] == 7.0).all()
        if dtype == torch.float16 and K == 131056:
            continue  # sums past its range
        check_linear(y[:M], xq, xs, w, ws)


@pytest.mark.parametrize("M", [2, 12, 70, 600])
def test_linear_strides(M):
    N, K = 77, 208
    xq, xs, w, ws = make_linear(M, N, K, M)
    wide = torch.full((M, K + 48), 55, dtype=torch.int8, device="cuda")
    wide[:, 16:16 + K] = xq.cuda()
    for pad, off in ((3, 1), (4, 4), (51, 0)):
        big = torch.full((M, N + pad + off), 7.0, dtype=torch.bfloat16, device="cuda")
        y = big[:, off:off + N]
        moe.moe_linear_i8(wide[:, 16:16 + K], xs.cuda(), w.cuda(), ws.cuda(), y)
        torch.cuda.synchronize()
        check_linear(y, xq, xs, w, ws)
        assert (big[:, :off] == 7.0).all() and (big[:, off + N:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 40])
def test_linear_largest_sums(M):
    """Rows of -128 over the longest axis: sums of 2^31 - 2^18, just inside int32."""
    N, K = 70, 131056
    one = torch.ones(max(M, N), device="cuda")
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_i8(xq, one[:M], w, one[:N], y)
    torch.cuda.synchronize()
    assert (y == float(2 ** 14 * K)).all()  # 2^18 * (2^13 - 1): exact in fp32


def test_quantize_then_linear():
    """The pair as a layer uses it, against the unquantised product: each
    quantised value is off by at most half a step."""
    M, N, K = 37, 200, 512
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    _, _, w, ws = make_linear(1, N, K, 4)
    q, s = quantize(x.cuda())
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_i8(q, s, w.cuda(), ws.cuda(), y)
    torch.cuda.synchronize()
    wd = w.double() * ws.double()[:, None]
    ref = x.double() @ wd.T
    step = x.double().abs().amax(dim=1, keepdim=True) / 127
    tol = 0.5 * step * wd.abs().sum(dim=1) + 8 * U32 * (x.double().abs() @ wd.abs().T)
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())


# ------------------------------------------------------------- expert FFN --

def make_bank(R, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    b = {"w13": torch.randint(-128, 128, (R, 2 * I, H), dtype=torch.int8, generator=g),
         "w2": torch.randint(-128, 128, (R, H, I), dtype=torch.int8, generator=g),
         "s13": (torch.rand(R, 2 * I, generator=g) + 0.5) / (73 * H ** 0.5),
         "s2": (torch.rand(R, H, generator=g) + 0.5) / (73 * I ** 0.5)}
    return b


def bank_on(b, where):
    if where == "device" or b["w13"].shape[0] == 0:
        t = {n: v.cuda() for n, v in b.items()}
        return moe.BankI8(t["w13"], t["s13"], t["w2"], t["s2"])
    t = {n: v if where == "host_weights" and n[0] == "s" else v.pin_memory() for n, v in b.items()}
    if where == "host_weights":
        return moe.BankI8(t["w13"], t["s13"].cuda(), t["w2"], t["s2"].cuda(),
                          moe.BANK_HOST_WEIGHTS)
    return moe.BankI8(t["w13"], t["s13"], t["w2"], t["s2"], moe.BANK_HOST)


def rows_of(b, owners):
    return {n: v[torch.as_tensor(np.asarray(owners)).long()] for n, v in b.items()}


def run_ffn(hot, cold, rm, ids, x, H, I, streams=False):
    T, k = ids.shape
    hs, cs = moe.Split.empty(hot.n_rows, T, k), moe.Split.empty(cold.n_rows, T, k)
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_route_split(ids.cuda(), torch.from_numpy(np.ascontiguousarray(rm, np.int32)).cuda(),
                        hot.n_rows, cold.n_rows, hs, cs, ninv)
    xq, xs = quantize(x.cuda())
    ws = torch.full((moe.moe_ffn_i8_workspace_bytes(T, k, H, I),), 0x7f, dtype=torch.uint8,
                    device="cuda")
    Y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream() if streams else None
    moe.moe_expert_ffn_i8(cold, cs, xq, xs, k, I, ws, Y, stream=side)
    moe.moe_expert_ffn_i8(hot, hs, xq, xs, k, I, ws, Y)
    torch.cuda.synchronize()
    return Y.cpu()


def check_ffn(Y, b, ids, x, H, I):
    T, k = ids.shape
    xq, xstep = layer_ref.quantize(x)
    Y = Y.view(T, k, H)
    # experts one by one, all their picks at once
    for e in torch.unique(ids).tolist():
        if not 0 <= e < b["w13"].shape[0]:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        s13, s2 = b["s13"][e].double(), b["s2"][e].double()
        gu = (xq[t] @ b["w13"][e].double().T) * xstep[t] * s13
        g, u = gu[:, :I], gu[:, I:]
        h = layer_ref.swiglu(g, u)
        dh = layer_ref.swiglu_bound(g, u, 4 * U32 * g.abs(), 4 * U32 * u.abs())
        hq, step = layer_ref.quantize(h)
        # an integer may turn where h's error reaches past half way
        most = 127 * step
        rel = dh.amax(dim=1, keepdim=True) / most.clamp_min(1e-300)
        r = 127 * h.abs() / most.clamp_min(1e-300)
        dr = 127 * dh / most.clamp_min(1e-300) + r * rel
        turn = ((r - r.floor() - 0.5).abs() <= 1.01 * dr).double()
        w2 = b["w2"][e].double()
        ref = (hq @ w2.T) * step * s2
        tol = (turn @ w2.abs().T) * step * s2
        tol = tol + (4 * U32 + 2 * rel + HALF_STEP[torch.bfloat16]) * (ref.abs() + tol)
        off = (Y[t, j].double() - ref).abs()
        assert bool((off <= tol + 1e-300).all()), (e, float((off / tol.clamp_min(1e-300)).max()))


FFN = [
    # T, k, E, H, I
    (1, 1, 1, 64, 64),
    (1, 2, 4, 256, 128),
    (7, 6, 12, 1024, 576),
    (16, 3, 4, 4096, 2880),    # experts with more than 8 slots: two units
    (5, 2, 6, 8192, 320),
    (3, 2, 3, 320, 8256),      # down axis past the streaming family
    (40, 4, 64, 192, 832),
    (130, 6, 16, 256, 192),    # tiles; part-filled ones
    (700, 2, 3, 128, 320),     # several tiles per expert
    (64, 32, 40, 64, 64),
    (4, 3, 4096, 64, 64),
]


@pytest.mark.parametrize("T,k,E,H,I", FFN)
def test_expert_ffn(T, k, E, H, I):
    b = make_bank(E, H, I, T + E)
    ids, _ = synth.gaussian_routing(T, k, E, 5)
    ids = torch.from_numpy(ids.astype(np.int32))
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    none = {n: v[:0] for n, v in b.items()}
    Y = run_ffn(bank_on(b, "device"), bank_on(none, "device"), np.arange(E), ids, x, H, I)
    check_ffn(Y, b, ids, x, H, I)


@pytest.mark.parametrize("T", [6, 150])
def test_ffn_bits_do_not_depend_on_the_banks(T):
    k, E, H, I = 4, 12, 512, 320
    b = make_bank(E, H, I, 3)
    ids, _ = synth.gaussian_routing(T, k, E, 7)
    ids = torch.from_numpy(ids.astype(np.int32))
    ids[0, 1], ids[T - 1] = -1, E + 5     # picks of no bank: their rows stay as they were
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    none = {n: v[:0] for n, v in b.items()}
    want = run_ffn(bank_on(b, "device"), bank_on(none, "device"), np.arange(E), ids, x, H, I)
    gone = (ids < 0) | (ids >= E)
    assert (want.view(T, k, H)[gone] == 7.0).all()
    check_ffn(want, b, ids, x, H, I)
    rm, ho, co = synth.random_map(E, 5, 4)
    for where in ("device", "host", "host_weights"):
        got = run_ffn(bank_on(rows_of(b, ho), "device"), bank_on(rows_of(b, co), where), rm, ids, x,
                      H, I, streams=True)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), where


def test_ffn_repeated_ids_and_special_tokens():
    T, k, E, H, I = 20, 3, 5, 128, 192
    b = make_bank(E, H, I, 9)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(2))
    ids[:, 2] = ids[:, 0]
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[4] = 0
    x[9, 7] = float("nan")
    none = {n: v[:0] for n, v in b.items()}
    Y = run_ffn(bank_on(b, "device"), bank_on(none, "device"), np.arange(E), ids, x, H, I)
    Yt = Y.view(T, k, H)
    assert torch.equal(Yt[:, 0].view(torch.int16), Yt[:, 2].view(torch.int16))
    assert (Yt[4] == 0).all() and Yt[9].isnan().all()
    keep = [t for t in range(T) if t != 9]
    check_ffn(Yt[keep].reshape(-1, H), b, ids[keep], x[keep], H, I)


@pytest.mark.parametrize("T", [8, 200])
def test_graph_replays_match_eager(T):
    k, E, H, I = 4, 16, 256, 320
    b = make_bank(E, H, I, 11)
    bank = bank_on(b, "device")
    rm = torch.arange(E, dtype=torch.int32, device="cuda")
    steps = []
    for s in range(4):
        ids, w = synth.gaussian_routing(T, k, E, 30 + s)
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16)
        steps.append([torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w).cuda(),
                      x.cuda()])
    st = [t.clone() for t in steps[0]]
    hs, cs = moe.Split.empty(E, T, k), moe.Split.empty(0, T, k)
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    xq = torch.empty(T, H, dtype=torch.int8, device="cuda")
    xs = torch.empty(T, device="cuda")
    ws = torch.empty(moe.moe_ffn_i8_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    shared = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    sw = torch.randint(-127, 128, (H, H), dtype=torch.int8, device="cuda")
    sws = torch.rand(H, device="cuda")

    def layer():  # the routed layer and a dense product of the same activations
        moe.moe_route_split(st[0], rm, E, 0, hs, cs, ninv)
        moe.moe_quantize_rows_i8(st[2], xq, xs)
        moe.moe_expert_ffn_i8(bank, hs, xq, xs, k, I, ws, Y)
        moe.moe_finalize(Y, st[1], out)
        moe.moe_linear_i8(xq, xs, sw, sws, shared)

    want = []
    for s in steps:
        for d, v in zip(st, s):
            d.copy_(v)
        layer()
        torch.cuda.synchronize()
        want.append((out.clone(), shared.clone()))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer()
    for rep in range(6):
        n = (rep * 3) % 4
        for d, v in zip(st, steps[n]):
            d.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip((out, shared), want[n]):
            assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
        assert torch.randn(64, 64, device="cuda").sum().isfinite()


@pytest.mark.parametrize("side", ["hot_stream", "cold_stream"])
def test_captured_layer_on_two_streams(side):
    """The whole int8 layer with a side stream, captured: the fork and the join
    are in the graph, and every replay gives the eager bits."""
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    T, k, E, H, I = 9, 3, 12, 256, 320
    b = make_bank(E, H, I, 17)
    rm, ho, co = synth.random_map(E, 4, 6)
    layer = ResidencyLayer(bank_on(rows_of(b, ho), "device"), bank_on(rows_of(b, co), "host"),
                           torch.from_numpy(rm.astype(np.int32)).cuda(), H, I)
    bufs = LayerBuffers.allocate(T, k, H, I, E - 4, 4, i8=True)
    other = torch.cuda.Stream()
    steps = []
    for s in range(3):
        ids, w = synth.gaussian_routing(T, k, E, 50 + s)
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16)
        steps.append([torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w).cuda(), x.cuda()])
    want = []
    for ids, w, x in steps:
        layer.forward(x.view(torch.uint16), ids, w, bufs)
        torch.cuda.synchronize()
        want.append(bufs.out.clone())
    st = [t.clone() for t in steps[0]]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer.forward(st[2], st[0], st[1], bufs, **{side: other})
    for rep in range(6):
        for d, v in zip(st, steps[rep % 3]):
            d.copy_(v)
        bufs.out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.out, want[rep % 3])
        assert torch.randn(64, 64, device="cuda").sum().isfinite()


def check_rows(y, rows, xq, xs, w, ws):
    for m in rows:
        for n in (0, 1, y.shape[1] // 2, y.shape[1] - 1):
            ref = float((xq[m].double() * w[n].double()).sum()) * float(xs[m]) * float(ws[n])
            assert abs(float(y[m, n]) - ref) <= (3.1 * U32 + HALF_STEP[y.dtype]) * abs(ref) + 2.0 ** -140, (m, n)


@pytest.mark.parametrize("M,N,K", [(3, 1100003, 4096), (20, 1100003, 4096), (70, 540001, 8192),
                                   (600001, 4090, 64), (2200003, 1000, 2048)])
def test_linear_offsets_past_32_bits(M, N, K):
    """Weights, outputs or activations of more than 4 GB."""
    g = torch.Generator(device="cuda").manual_seed(M)
    xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(M, device="cuda", generator=g) + 0.5
    ws = (torch.rand(N, device="cuda", generator=g) + 0.5) / 1000
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert max(w.numel(), 2 * y.numel(), xq.numel()) > 2 ** 32
    moe.moe_linear_i8(xq, xs, w, ws, y)
    torch.cuda.synchronize()
    check_rows(y, (0, 1, M // 2, M - 2, M - 1), xq, xs, w, ws)


def test_layers_of_no_tokens():
    """Steps of no tokens, in each form of the layer, launch nothing that fails."""
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    k, E, H, I = 2, 4, 128, 64
    b = make_bank(E, H, I, 3)
    rm = torch.tensor([0, 1, -1, -2], dtype=torch.int32, device="cuda")
    mx = [torch.zeros(s, dtype=torch.uint8, device="cuda")
          for s in ((2, 2 * I, H // 2), (2, 2 * I, H // 32), (2, H, I // 2), (2, H, I // 32))]
    ids, w = torch.empty(0, k, dtype=torch.int32, device="cuda"), torch.empty(0, k, device="cuda")
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    i8 = [bank_on({n: v[i:i + 2] for n, v in b.items()}, where) for i, where in ((0, "device"), (2, "host"))]
    for layer, kind in ((ResidencyLayer(*i8, rm, H, I), True),
                        (ResidencyLayer(moe.Bank(*mx), moe.Bank(*mx), rm, H, I), False)):
        bufs = LayerBuffers.allocate(0, k, H, I, 2, 2, i8=kind)
        bufs.out.fill_(7)
        layer.route(torch.empty(0, E, device="cuda"), ids, w)
        layer.forward(x, ids, w, bufs)
        if not kind:
            layer.forward_few(x, ids, w, bufs)
        torch.cuda.synchronize()
        assert (bufs.out == 7).all()
