"""The 8-bit floating point products against their 64-bit forms: quantised rows
exactly, the dense product within its fp32 sums and the output's rounding, the
expert FFN within what the fp32 errors of h can turn in its quantisation; strides,
odd sizes, special values, banks, streams and HIP graphs."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import f8_ref
import synth
from f8_ref import blocks
from layer_ref import HALF_STEP, U32

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def quantize(x, stream=None):
    rows, K = x.shape
    q = torch.full((rows + 1, K), 99, dtype=torch.uint8, device="cuda").view(F8)
    s = torch.full((rows + 1, blocks(K)), 99.0, device="cuda")
    torch.cuda.synchronize()
    moe.moe_quantize_rows_f8(x, q[:rows], s[:rows], stream=stream)
    torch.cuda.synchronize()
    assert (q[rows].view(torch.uint8) == 99).all() and (s[rows] == 99.0).all()
    return q[:rows], s[:rows]


def check_quantize(x):
    q, s = quantize(x)
    rq, most = f8_ref.quantize(x.cpu().float())
    assert torch.equal(f8_ref.values(q), rq)
    # one fp32 division, rounded to nearest by both
    assert np.array_equal(s.cpu().numpy(), most[:, ::128].float().numpy() / np.float32(448))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 8), (2, 16), (9, 100), (4, 128), (3, 129), (33, 136),
                                    (17, 256), (6, 512), (2, 2048), (7, 4096), (1, 4104), (2, 8200),
                                    (1, 131072), (70, 2880), (66000, 24)])
def test_quantize_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * 131 + K)
    x = (torch.randn(rows, K, generator=g) * torch.logspace(-3, 3, rows)[:, None]).to(dtype)
    check_quantize(x.cuda())


def test_quantize_many_rows_of_many_blocks():
    """Rows enough that one workgroup takes all blocks of a row."""
    x = torch.randn(66000, 2200, device="cuda").to(torch.bfloat16)
    q, s = quantize(x)
    for part in (slice(0, 3), slice(40000, 40003), slice(65997, 66000)):
        rq, most = f8_ref.quantize(x[part].cpu().float())
        assert torch.equal(f8_ref.values(q[part]), rq)
        assert torch.equal(s[part].cpu(), most[:, ::128].float() / 448)


def test_quantize_ties_and_borders():
    """Every middle between two E4M3 values, its two fp32 neighbours, and the values
    themselves, of both signs, at several magnitudes."""
    mid = ((f8_ref.GRID[1:] + f8_ref.GRID[:-1]) / 2).float()
    all_ = torch.cat([f8_ref.GRID.float(), mid, torch.nextafter(mid, torch.tensor(1e9)),
                      torch.nextafter(mid, torch.tensor(0.0))])
    all_ = torch.cat([all_, -all_])
    pad = torch.zeros(-all_.numel() % 127)
    rows = torch.cat([all_, pad]).view(-1, 127)
    x = torch.cat([torch.full((rows.shape[0], 1), 448.0), rows], dim=1)
    for f in (1.0, 2.0 ** -60, 2.0 ** 100, 3.0, 0.7):  # 3: middles stay exact for fewer bits
        check_quantize((x * f).cuda())
        check_quantize((x * f)[:, 1:].cuda())      # odd rows: the elementwise form, another largest value
    for f in (1.0, 2.0 ** -5):
        check_quantize((x * f).half().cuda())
        check_quantize((x * f).bfloat16().cuda())
    q, _ = quantize(x[:1].cuda())
    t = torch.zeros(1, 128)
    t[0, :6] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10])
    q, _ = quantize(t.cuda())
    assert f8_ref.values(q)[0, :6].tolist() == [448.0, 16.0, 20.0, -16.0, 0.0, 2.0 ** -8]


def test_quantize_strides_and_offsets():
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(6, 403, generator=g).cuda()
    check_quantize(wide[:, 1:298])          # rows 4 bytes off a 16-byte boundary
    check_quantize(wide.half()[:, :200])    # vectors' length, unaligned row stride
    check_quantize(wide[::2, :300])
    flat = torch.zeros(2 * 2 ** 30 + 64, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((3, 64), (2 ** 30, 1))  # the third row 4 GB on
    far.copy_(torch.randn(3, 64, generator=g).to(torch.bfloat16))
    check_quantize(far)


def test_quantize_special_blocks():
    x = torch.randn(7, 256, generator=torch.Generator().manual_seed(6))
    x[0, :128] = 0.0
    x[1, 5] = float("inf")
    x[2, 255] = float("nan")
    x[3, 128:] *= 1e-40               # the scale would be subnormal
    x[4, 0] = torch.finfo(torch.float32).max
    x[5] = -0.0
    q, s = quantize(x.cuda())
    z = f8_ref.values(q)
    for r, b in ((0, 0), (1, 0), (2, 1), (3, 1), (5, 0), (5, 1)):
        assert (z[r, 128 * b:128 * b + 128] == 0).all()
    assert s[0, 0] == 0 and s[3, 1] == 0 and (s[5] == 0).all() and s[1, 0].isnan() and s[2, 1].isnan()
    assert s[1, 1].isfinite() and s[2, 0].isfinite()
    check_quantize(x[[4, 6]].cuda())
    y = torch.empty(7, 8, device="cuda")
    w = torch.ones(8, 256, device="cuda").to(F8)
    moe.moe_linear_f8(q, s, w, torch.ones(1, 2, device="cuda"), y)
    torch.cuda.synchronize()
    assert y[[1, 2]].isnan().all() and (y[5] == 0).all() and y[[0, 3, 6]].isfinite().all()


def make_linear(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)

    def codes(r, c):  # every finite code
        b = torch.randint(0, 254, (r, c), dtype=torch.uint8, generator=g)
        return (b + (b >= 127).to(torch.uint8)).view(F8)
    xs = torch.rand(M, blocks(K), generator=g) + 0.01
    ws = (torch.rand(blocks(N), blocks(K), generator=g) + 0.01) / (1e4 * K ** 0.5)
    return codes(M, K), xs, codes(N, K), ws


def check_linear(y, xq, xs, w, ws):
    ref, off = f8_ref.product(f8_ref.values(xq), xs, f8_ref.values(w), ws, y.dtype)
    # ... then the type's rounding, and fp16's subnormals
    tol = off + HALF_STEP[y.dtype] * (ref.abs() + off) + (2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -140)
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


LINEAR = [(1, 1, 16), (1, 7, 32), (1, 5760, 4096), (3, 100, 2880), (8, 64, 1024), (9, 63, 1040),
          (16, 333, 4096), (16, 40, 8192), (2, 24, 8208), (17, 65, 128), (64, 64, 64),
          (100, 130, 272), (257, 511, 1040), (33, 4096, 2880), (1001, 2047, 1040),
          (4095, 4100, 144), (300, 257, 16), (5, 3, 131072), (700, 1500, 2064), (129, 8200, 400)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K):
    xq, xs, w, ws = make_linear(M, N, K, M + N + K)
    for dtype in TYPES:
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        moe.moe_linear_f8(xq.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y[:M])
        torch.cuda.synchronize()
        assert (y[M] == 7.0).all()
        check_linear(y[:M], xq, xs, w, ws)


@pytest.mark.parametrize("M", [2, 12, 70, 600])
def test_linear_strides(M):
    N, K = 77, 208
    xq, xs, w, ws = make_linear(M, N, K, M)
    wide = torch.full((M, K + 48), 0x7f, dtype=torch.uint8, device="cuda").view(F8)  # NaN around the rows
    wide.view(torch.uint8)[:, 16:16 + K] = xq.cuda().view(torch.uint8)
    for pad, off in ((3, 1), (4, 4), (51, 0)):
        big = torch.full((M, N + pad + off), 7.0, dtype=torch.bfloat16, device="cuda")
        y = big[:, off:off + N]
        moe.moe_linear_f8(wide[:, 16:16 + K], xs.cuda(), w.cuda(), ws.cuda(), y)
        torch.cuda.synchronize()
        check_linear(y, xq, xs, w, ws)
        assert (big[:, :off] == 7.0).all() and (big[:, off + N:] == 7.0).all()


@pytest.mark.parametrize("M,N", [(1, 300), (40, 300), (600, 600), (2100, 8200)])
def test_linear_special_values(M, N):
    """A NaN code or scale reaches the outputs that read it and no others; an
    infinite scale of the last, part-filled block gives infinities."""
    K = 400
    xq, xs, w, ws = make_linear(M, N, K, 9)
    w.view(torch.uint8)[:, 399] = 0x38  # 1.0
    xq.view(torch.uint8)[:, 384:] = 0x38
    w.view(torch.uint8)[:, 384:] = 0x38
    base = torch.empty(M, N, device="cuda")
    moe.moe_linear_f8(xq.cuda(), xs.cuda(), w.cuda(), ws.cuda(), base)
    bad_w, bad_s = w.clone(), ws.clone()
    bad_w.view(torch.uint8)[5, 130] = 0x7f
    bad_w.view(torch.uint8)[200, 399] = 0xff
    bad_s[blocks(N) - 1, 3] = float("inf")
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_f8(xq.cuda(), xs.cuda(), bad_w.cuda(), bad_s.cuda(), y)
    torch.cuda.synchronize()
    last = 128 * (blocks(N) - 1)
    keep = [n for n in range(last) if n not in (5, 200)]
    assert y[:, 5].isnan().all() and y[:, 200].isnan().all()
    assert torch.equal(y[:, keep], base[:, keep])
    assert (y[:, last:] == float("inf")).all()


def test_quantize_then_linear():
    """The pair as a layer uses it, against the unquantised product: each quantised
    value is off by at most half a step of its size or of the smallest one."""
    M, N, K = 37, 200, 500
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    K = 496
    x = x[:, :K].contiguous()
    _, _, w, ws = make_linear(1, N, K, 4)
    q, s = quantize(x.cuda())
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_f8(q, s, w.cuda(), ws.cuda(), y)
    torch.cuda.synchronize()
    wd = f8_ref.values(w) * f8_ref.spread(ws, N, K)
    xd = x.double()
    _, most = f8_ref.quantize(x.float())
    half = torch.maximum(xd.abs() * 2.0 ** -4, most / 448 * 2.0 ** -10)
    tol = half @ wd.abs().T + 300 * U32 * ((xd.abs() + half) @ wd.abs().T)
    assert bool(((y.cpu().double() - xd @ wd.T).abs() <= tol).all())


# ------------------------------------------------------------- expert FFN --

def make_bank(R, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    b = {n: (torch.randn(s, generator=g) * 112).clamp(-448, 448).to(F8)
         for n, s in (("w13", (R, 2 * I, H)), ("w2", (R, H, I)))}
    b["s13"] = (torch.rand(R, 2, blocks(I), blocks(H), generator=g) + 0.5) / (112 * H ** 0.5)
    b["s2"] = (torch.rand(R, blocks(H), blocks(I), generator=g) + 0.5) / (112 * I ** 0.5)
    return b


def rows_of(b, owners):
    at = torch.as_tensor(np.asarray(owners)).long()
    return {n: v.view(torch.uint8)[at].view(F8) if v.dtype == F8 else v[at] for n, v in b.items()}


def bank_on(b, where):
    if where == "device" or b["w13"].shape[0] == 0:
        t = {n: v.cuda() for n, v in b.items()}
        return moe.BankF8(t["w13"], t["s13"], t["w2"], t["s2"])
    t = {n: v if where == "host_weights" and n[0] == "s" else v.pin_memory() for n, v in b.items()}
    if where == "host_weights":
        return moe.BankF8(t["w13"], t["s13"].cuda(), t["w2"], t["s2"].cuda(), moe.BANK_HOST_WEIGHTS)
    return moe.BankF8(t["w13"], t["s13"], t["w2"], t["s2"], moe.BANK_HOST)


def run_ffn(hot, cold, rm, ids, x, H, I, streams=False):
    T, k = ids.shape
    hs, cs = moe.Split.empty(hot.n_rows, T, k), moe.Split.empty(cold.n_rows, T, k)
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_route_split(ids.cuda(), torch.from_numpy(np.ascontiguousarray(rm, np.int32)).cuda(),
                        hot.n_rows, cold.n_rows, hs, cs, ninv)
    xq, xs = quantize(x.cuda())
    ws = torch.full((moe.moe_ffn_f8_workspace_bytes(T, k, H, I),), 0x7f, dtype=torch.uint8, device="cuda")
    Y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream() if streams else None
    moe.moe_expert_ffn_f8(cold, cs, xq, xs, k, I, ws, Y, stream=side)
    moe.moe_expert_ffn_f8(hot, hs, xq, xs, k, I, ws, Y)
    torch.cuda.synchronize()
    return Y.cpu()


def check_ffn(Y, b, ids, x, H, I):
    T, k = ids.shape
    Y = Y.view(T, k, H)
    for e in torch.unique(ids).tolist():
        if not 0 <= e < b["w13"].shape[0]:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        ref, tol = f8_ref.ffn(x[t].float(), b, e)
        err = (Y[t, j].double() - ref).abs()
        assert bool((err <= tol + 1e-300).all()), (e, float((err / tol.clamp_min(1e-300)).max()))


FFN = [
    # T, k, E, H, I
    (1, 1, 1, 64, 64),
    (1, 2, 4, 256, 128),
    (7, 6, 12, 1024, 576),
    (16, 3, 4, 4096, 2880),
    (5, 2, 6, 8192, 320),
    (3, 2, 3, 320, 8256),
    (40, 4, 64, 192, 832),
    (130, 6, 16, 256, 192),    # part-filled tiles
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


def test_ffn_refuses_a_split_of_too_few_entries():
    T, k, E, H, I = 6, 2, 8, 128, 64
    b = bank_on(make_bank(E, H, I, 1), "device")
    xq = torch.zeros(T, H, dtype=F8, device="cuda")
    xs = torch.zeros(T, 1, dtype=torch.float32, device="cuda")
    ws = torch.zeros(moe.moe_ffn_f8_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    Y = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    for made_for in ((E, 2, k), (3, T, k)):
        with pytest.raises(moe.MoeError, match="split"):
            moe.moe_expert_ffn_f8(b, moe.Split.empty(*made_for), xq, xs, k, I, ws, Y)
    moe.moe_expert_ffn_f8(b, moe.Split.empty(E, T, k), xq, xs, k, I, ws, Y)  # of no picks


def test_ffn_of_no_valid_picks():
    T, k, E, H, I = 9, 2, 4, 128, 128
    b = make_bank(E, H, I, 9)
    none = {n: v[:0] for n, v in b.items()}
    ids = torch.full((T, k), -1, dtype=torch.int32)
    Y = run_ffn(bank_on(b, "device"), bank_on(none, "device"), np.arange(E), ids,
                torch.ones(T, H, dtype=torch.bfloat16), H, I)
    assert (Y == 7.0).all()


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
        steps.append([torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w).cuda(), x.cuda()])
    st = [t.clone() for t in steps[0]]
    hs, cs = moe.Split.empty(E, T, k), moe.Split.empty(0, T, k)
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    xq = torch.empty(T, H, dtype=F8, device="cuda")
    xs = torch.empty(T, blocks(H), device="cuda")
    ws = torch.empty(moe.moe_ffn_f8_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    shared = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    sw = torch.randn(H, H, device="cuda").to(F8)
    sws = torch.rand(blocks(H), blocks(H), device="cuda")

    def layer():  # the routed layer and a dense product of the same activations
        moe.moe_route_split(st[0], rm, E, 0, hs, cs, ninv)
        moe.moe_quantize_rows_f8(st[2], xq, xs)
        moe.moe_expert_ffn_f8(bank, hs, xq, xs, k, I, ws, Y)
        moe.moe_finalize(Y, st[1], out)
        moe.moe_linear_f8(xq, xs, sw, sws, shared)

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
    """ResidencyLayer on FP8 banks with a side stream, captured: gate logits to the
    output, every replay the eager bits, and those the rows' weighted sums."""
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    T, k, E, H, I = 9, 3, 12, 256, 320
    b = make_bank(E, H, I, 17)
    rm, ho, co = synth.random_map(E, 4, 6)
    layer = ResidencyLayer(bank_on(rows_of(b, ho), "device"), bank_on(rows_of(b, co), "host"),
                           torch.from_numpy(rm.astype(np.int32)).cuda(), H, I)
    bufs = LayerBuffers.allocate(T, k, H, I, E - 4, 4, f8=True)
    other = torch.cuda.Stream()
    steps = []
    for s in range(3):
        g = torch.Generator().manual_seed(s)
        steps.append([torch.randn(T, E, generator=g).cuda(), torch.randn(T, H, generator=g).bfloat16().cuda()])
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    want = []
    for logits, x in steps:
        layer.route(logits, ids, w)
        layer.forward(x.view(torch.uint16), ids, w, bufs)
        torch.cuda.synchronize()
        want.append(bufs.out.clone())
        ref = torch.zeros(T, H, dtype=torch.float64)
        tol = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                y, off = f8_ref.ffn(x[t:t + 1].cpu().float(), b, int(ids[t, j]))
                ref[t] += float(w[t, j]) * y[0]
                tol[t] += float(w[t, j]) * (off[0] + 2 * k * U32 * y[0].abs())
        tol += HALF_STEP[torch.bfloat16] * (ref.abs() + tol)
        assert bool(((bufs.out.view(torch.bfloat16).cpu().double() - ref).abs() <= tol).all())
    st = [t.clone() for t in steps[0]]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer.route(st[0], ids, w)
        layer.forward(st[1], ids, w, bufs, **{side: other})
    for rep in range(6):
        for d, v in zip(st, steps[rep % 3]):
            d.copy_(v)
        bufs.out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.out, want[rep % 3])
        assert torch.randn(64, 64, device="cuda").sum().isfinite()


def test_two_calls_at_once():
    """Two steps on two streams, each with buffers of its own."""
    T, k, E, H, I = 60, 2, 8, 256, 192
    b = make_bank(E, H, I, 21)
    bank = bank_on(b, "device")
    runs = []
    for s in range(2):
        ids, _ = synth.gaussian_routing(T, k, E, 60 + s)
        ids = torch.from_numpy(ids.astype(np.int32))
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16)
        hs, cs = moe.Split.empty(E, T, k), moe.Split.empty(0, T, k)
        moe.moe_route_split(ids.cuda(), torch.arange(E, dtype=torch.int32, device="cuda"), E, 0, hs, cs,
                            torch.zeros(1, dtype=torch.int32, device="cuda"))
        runs.append((ids, x, hs, quantize(x.cuda()), torch.cuda.Stream(),
                     torch.empty(moe.moe_ffn_f8_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda"),
                     torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for ids, x, hs, (xq, xs), stream, ws, Y in runs:
            moe.moe_expert_ffn_f8(bank, hs, xq, xs, k, I, ws, Y, stream=stream)
    torch.cuda.synchronize()
    for ids, x, _, _, _, _, Y in runs:
        check_ffn(Y.cpu(), b, ids, x, H, I)


def check_rows(y, rows, xq, xs, w, ws):
    N = y.shape[1]
    for n in (0, 1, N // 2, N - 1):
        at = list(rows)
        ref, off = f8_ref.product(f8_ref.values(xq[at]), xs[at].cpu(), f8_ref.values(w[n:n + 1]),
                                  ws[n // 128:n // 128 + 1].cpu(), y.dtype)
        tol = off + HALF_STEP[y.dtype] * (ref.abs() + off) + 2.0 ** -140
        assert bool(((y[at, n:n + 1].cpu().double() - ref).abs() <= tol).all()), n


@pytest.mark.parametrize("M,N,K", [(3, 1100003, 4096), (20, 1100003, 4096), (70, 540001, 8192),
                                   (600001, 4090, 64), (2200003, 1000, 2048)])
def test_linear_offsets_past_32_bits(M, N, K):
    """Weights, outputs or activations of more than 4 GB."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def codes(r, c):  # finite codes below 16
        return torch.randint(0, 90, (r, c), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    xq, w = codes(M, K), codes(N, K)
    xs = torch.rand(M, blocks(K), device="cuda", generator=g) + 0.5
    ws = (torch.rand(blocks(N), blocks(K), device="cuda", generator=g) + 0.5) / 1000
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert max(w.numel(), 2 * y.numel(), xq.numel()) > 2 ** 32
    moe.moe_linear_f8(xq, xs, w, ws, y)
    torch.cuda.synchronize()
    check_rows(y, (0, 1, M // 2, M - 2, M - 1), xq, xs, w, ws)


def test_layers_of_no_tokens():
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    k, E, H, I = 2, 4, 128, 64
    b = make_bank(E, H, I, 3)
    rm = torch.tensor([0, 1, -1, -2], dtype=torch.int32, device="cuda")
    layer = ResidencyLayer(bank_on(rows_of(b, [0, 1]), "device"), bank_on(rows_of(b, [2, 3]), "host"), rm, H, I)
    bufs = LayerBuffers.allocate(0, k, H, I, 2, 2, f8=True)
    bufs.out.fill_(7)
    ids, w = torch.empty(0, k, dtype=torch.int32, device="cuda"), torch.empty(0, k, device="cuda")
    layer.forward(torch.empty(0, H, dtype=torch.bfloat16, device="cuda"), ids, w, bufs)
    torch.cuda.synchronize()
    assert (bufs.out == 7).all()
