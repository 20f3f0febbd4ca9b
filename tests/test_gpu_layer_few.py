"""moe_layer_few_mxfp4 (the whole layer for a few tokens in two launches)
against the 64-bit form, elementwise within the derived bound; its bits across
bank placements; padding, repeated and invalid ids; the counter; streams and
HIP graphs."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import layer_ref
import synth
from gpu_util import REL_L2, device_bank, empty_bank_host, host_bank, pinned_bank

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def bank_on(arrays, where):
    if where == "device" or arrays["w13"].shape[0] == 0:
        return device_bank(arrays)
    b = pinned_bank(arrays)
    if where == "host_weights":
        b = moe.Bank(b.w13, b.s13.cuda(), b.w2, b.s2.cuda(), on_host=moe.BANK_HOST_WEIGHTS)
    return b


def make_step(T, k, E, H, I, n_cold, seed, pads=0, repeat=False):
    rm, ho, co = synth.random_map(E, n_cold, seed)
    # scale bytes 2^-9 .. 2^-6: gate and up values of order one, so that the
    # SwiGLU is neither linear nor saturated
    arr = {n: host_bank(o, seed, 0, H, I, scale_lo=118, scale_cnt=4)
           for n, o in (("hot", ho), ("cold", co))}
    ids, w = synth.gaussian_routing(T, k, E, seed)
    ids = ids.copy()
    if repeat:  # the same expert at two places of a token, weights of their own
        ids[:, k - 1] = ids[:, 0]
    if pads:
        ids[T - pads:] = -1
    x = torch.from_numpy(synth.activations(T, H, seed).view(np.int16)).view(torch.bfloat16)
    return rm, arr, torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w), x


def run(arr, rm, ids, w, x, H, I, where=("device", "device"), stream=None, counts=None,
        count_tmax=256):
    T, k = ids.shape
    hot, cold = bank_on(arr["hot"], where[0]), bank_on(arr["cold"], where[1])
    ws = torch.full((moe.moe_layer_few_workspace_bytes(T, k, H, I),), 0x7f, dtype=torch.uint8,
                    device="cuda")
    out = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ninv = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    rmd = torch.from_numpy(np.ascontiguousarray(rm, np.int32)).cuda()
    torch.cuda.synchronize()
    moe.moe_layer_few_mxfp4(hot, cold, rmd, x.cuda(), ids.cuda(), w.cuda(), I, ws, out[:T], ninv,
                            counts_layer=counts, count_tmax=count_tmax, stream=stream)
    torch.cuda.synchronize()
    assert (out[T] == 7.0).all()  # the row behind the last token
    return out[:T].cpu(), int(ninv)


def row_of(rm, n_hot, n_cold):
    def f(e):
        if not 0 <= e < len(rm):
            return None
        m = int(rm[e])
        at = ("hot", m) if m >= 0 else ("cold", -1 - m)
        return at if at[1] < (n_hot if m >= 0 else n_cold) else None
    return f


def check(got, ref, bound):
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound.clamp_min(1e-300)).max())
    # two independent roundings to bf16 (h and out): 2^-8 * sqrt(2) = 5.5e-3 at most
    assert float(off.norm() / ref.norm().clamp_min(1e-300)) <= REL_L2


SHAPES = [
    # T, k, E, H, I, cold experts
    (1, 1, 1, 64, 64, 0),
    (1, 2, 4, 256, 128, 1),
    (7, 6, 24, 4096, 2880, 3),
    (16, 6, 20, 4096, 2880, 2),
    (8, 3, 12, 320, 192, 4),       # both axes end inside a chunk
    (9, 2, 5, 2112, 576, 2),       # two chunks per wavefront, ragged; a second token set
    (16, 8, 16, 1024, 4096, 16),   # everything cold; the longest I
    (5, 4, 9, 8192, 64, 3),        # the longest H
    (16, 2, 6, 4160, 832, 0),      # four chunks per wavefront, ragged
    (16, 32, 40, 256, 128, 7),     # 512 picks: several phases of h rows
    (16, 32, 32, 64, 2112, 0),     # every token picks every expert
    (3, 5, 4096, 64, 64, 40),      # the largest expert count
]


@pytest.mark.parametrize("T,k,E,H,I,n_cold", SHAPES)
def test_against_64_bits(T, k, E, H, I, n_cold):
    rm, arr, ids, w, x = make_step(T, k, E, H, I, n_cold, 3)
    out, ninv = run(arr, rm, ids, w, x, H, I)
    ref, bound, bad = layer_ref.layer(arr, row_of(rm, E - n_cold, n_cold), x, ids, w, H, I)
    assert ninv == bad == 0
    check(out, ref, bound)


@pytest.mark.parametrize("T,k,E,H,I", [(7, 4, 12, 1024, 576), (16, 3, 10, 320, 1088),
                                       (3, 2, 6, 8192, 128), (9, 2, 6, 4160, 256),
                                       (5, 4, 7, 64, 64), (7, 3, 7, 4096, 2880),
                                       (9, 2, 6, 8192, 64), (16, 3, 6, 64, 4096)])
def test_bits_do_not_depend_on_the_banks(T, k, E, H, I):
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 4, 5)
    want, _ = run(arr, rm, ids, w, x, H, I)
    for where in (("device", "host"), ("device", "host_weights"), ("host", "device"),
                  ("host", "host")):
        got, _ = run(arr, rm, ids, w, x, H, I, where)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), where
    all_map, owner, _ = synth.all_hot_map(E)
    one = {"hot": host_bank(owner, 5, 0, H, I, scale_lo=118, scale_cnt=4),
           "cold": {n: v[:0] for n, v in arr["cold"].items()}}
    got, _ = run(one, all_map, ids, w, x, H, I)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_padding_repeated_and_invalid_ids():
    T, k, E, H, I = 11, 4, 10, 512, 320
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 3, 7, pads=2, repeat=True)
    x[T - 1] = float("nan")        # what a padding token holds reaches no one
    ids[0, 1] = E                  # outside the experts
    ids[1, 2] = -2147483648
    rm = rm.copy()
    rm[int(ids[2, 0])] = 99        # a row outside its bank
    ref, bound, bad = layer_ref.layer(arr, row_of(rm, E - 3, 3), x.nan_to_num(0), ids, w, H, I)
    out, ninv = run(arr, rm, ids, w, x, H, I)
    assert ninv == bad > 2 * k
    assert (out[T - 2:] == 0).all()
    check(out, ref, bound)


def test_all_picks_invalid():
    T, k, E, H, I = 4, 2, 6, 256, 128
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 2, 9, pads=4)
    out, ninv = run(arr, rm, ids, w, x, H, I)
    assert ninv == T * k and (out == 0).all()


def test_infinite_expert_reaches_its_own_tokens_only():
    T, k, E, H, I = 6, 2, 8, 256, 256
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 2, 11)
    for t in range(T):
        ids[t] = torch.tensor([t % 3, 3 + t % 4], dtype=torch.int32)
    at = row_of(rm, E - 2, 2)(int(ids[0, 0]))
    for n in ("s13", "s2"):
        arr[at[0]][n][at[1]] = 255  # NaN scales
    out, _ = run(arr, rm, ids, w, x, H, I)
    hit = (ids == ids[0, 0]).any(dim=1)
    assert out[hit].isnan().all() and out[~hit].isfinite().all()
    keep = [t for t in range(T) if not hit[t]]
    ref, bound, _ = layer_ref.layer(arr, row_of(rm, E - 2, 2), x[keep], ids[keep], w[keep], H, I)
    check(out[keep], ref, bound)


def test_counter():
    T, k, E, H, I = 16, 4, 12, 128, 64
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 3, 13, pads=3)
    counts = torch.arange(E, dtype=torch.int32, device="cuda")
    run(arr, rm, ids, w, x, H, I, counts=counts)
    want = np.arange(E) + np.bincount(ids[ids >= 0].numpy(), minlength=E)
    assert np.array_equal(counts.cpu().numpy(), want)
    run(arr, rm, ids, w, x, H, I, counts=counts, count_tmax=T - 1)  # a step too large to count
    assert np.array_equal(counts.cpu().numpy(), want)


def test_agrees_with_the_split_path():
    from gpu_util import run_layer
    T, k, E, H, I = 7, 4, 16, 1024, 1536
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 5, 15)
    out, _ = run(arr, rm, ids, w, x, H, I)
    _, split, _ = run_layer(device_bank(arr["hot"]), pinned_bank(arr["cold"]), rm, ids.numpy(),
                            w.numpy(), x.view(torch.int16).numpy().view(np.uint16), H, I)
    split = torch.from_numpy(split.view(np.int16)).view(torch.bfloat16).double()
    # each is within its roundings of the same value
    assert float((out.double() - split).norm() / split.norm()) <= 2 * REL_L2


def test_graph_replays_match_eager():
    """Two captured graphs with a workspace each, replayed in turn with eager
    work between, on inputs copied in."""
    T, k, E, H, I = 8, 4, 16, 1024, 576
    steps = [make_step(T, k, E, H, I, 4, 21)]
    rm, arr = steps[0][:2]
    for s in (22, 23, 24):
        _, _, ids, w, x = make_step(T, k, E, H, I, 4, s)
        steps.append((rm, arr, ids, w, x))
    want = [run(arr, rm, i, w, x, H, I)[0] for _, _, i, w, x in steps]
    hot, cold = device_bank(arr["hot"]), pinned_bank(arr["cold"])
    rmd = torch.from_numpy(rm.astype(np.int32)).cuda()
    graphs = []
    for _ in range(2):
        st = [t.cuda() for t in steps[0][2:]]
        ws = torch.empty(moe.moe_layer_few_workspace_bytes(T, k, H, I), dtype=torch.uint8,
                         device="cuda")
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
        counts = torch.zeros(E, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            moe.moe_layer_few_mxfp4(hot, cold, rmd, st[2], st[0], st[1], I, ws, out, ninv,
                                    counts_layer=counts)
        graphs.append((g, st, out, counts))
    for rep in range(6):
        a, b = rep % 4, (rep + 1) % 4
        for (g, st, _, _), n in zip(graphs, (a, b)):
            for dst, src in zip(st, steps[n][2:]):
                dst.copy_(src)
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, _, out, _), n in zip(graphs, (a, b)):
            assert torch.equal(out.cpu().view(torch.int16), want[n].view(torch.int16))
        assert torch.randn(100, 100, device="cuda").sum().isfinite()
    assert int(graphs[0][3].sum()) == 6 * T * k


def test_two_calls_at_once_on_two_streams():
    T, k, E, H, I = 16, 4, 16, 1024, 576
    rm, arr, ids, w, x = make_step(T, k, E, H, I, 4, 31)
    want, _ = run(arr, rm, ids, w, x, H, I)
    hot, cold = device_bank(arr["hot"]), device_bank(arr["cold"])
    rmd, idd, wd, xd = (torch.from_numpy(rm.astype(np.int32)).cuda(), ids.cuda(), w.cuda(), x.cuda())
    calls = []
    for _ in range(2):
        calls.append((torch.cuda.Stream(),
                      torch.empty(moe.moe_layer_few_workspace_bytes(T, k, H, I), dtype=torch.uint8,
                                  device="cuda"),
                      torch.empty(T, H, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(1, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws, out, ninv in calls:
            moe.moe_layer_few_mxfp4(hot, cold, rmd, xd, idd, wd, I, ws, out, ninv, stream=s)
    torch.cuda.synchronize()
    for _, _, out, _ in calls:
        assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


def test_residency_layer_runs_gate_few_and_i8():
    """ResidencyLayer: router logits through route, then forward_few, forward and
    (with 8-bit banks) the int8 forward on one or two streams."""
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    T, k, E, H, I = 7, 3, 12, 512, 320
    rm, arr, _, _, x = make_step(T, k, E, H, I, 4, 41)
    rmd = torch.from_numpy(rm.astype(np.int32)).cuda()
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    layer = ResidencyLayer(device_bank(arr["hot"]), pinned_bank(arr["cold"]), rmd, H, I)
    bufs = LayerBuffers.allocate(T, k, H, I, E - 4, 4)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    xd = x.cuda()
    layer.route(logits.cuda(), ids, w)
    layer.forward_few(xd, ids, w, bufs)
    torch.cuda.synchronize()
    few = bufs.out[:T].cpu().view(torch.bfloat16)
    ref, bound, _ = layer_ref.layer(arr, row_of(rm, E - 4, 4), x, ids.cpu(), w.cpu(), H, I)
    check(few, ref, bound)
    layer.forward(xd, ids, w, bufs)
    torch.cuda.synchronize()
    full = bufs.out[:T].cpu().view(torch.bfloat16).double()
    assert float((full - few.double()).norm() / full.norm()) <= 2 * REL_L2

    g = torch.Generator().manual_seed(2)
    rows = {"w13": torch.randint(-127, 128, (E, 2 * I, H), dtype=torch.int8, generator=g),
            "s13": torch.rand(E, 2 * I, generator=g) / (73 * H ** 0.5),
            "w2": torch.randint(-127, 128, (E, H, I), dtype=torch.int8, generator=g),
            "s2": torch.rand(E, H, generator=g) / (73 * I ** 0.5)}
    # row of an expert in either bank
    hot = {n: torch.empty_like(v[:E - 4]) for n, v in rows.items()}
    cold = {n: torch.empty_like(v[:4]).pin_memory() for n, v in rows.items()}
    for e in range(E):
        for n in rows:
            (hot if rm[e] >= 0 else cold)[n][rm[e] if rm[e] >= 0 else -1 - rm[e]] = rows[n][e]
    mk = lambda b, where, on: moe.BankI8(*(where(b[n]) for n in ("w13", "s13", "w2", "s2")), on)  # noqa: E731
    i8 = ResidencyLayer(mk(hot, lambda t: t.cuda(), moe.BANK_DEVICE),
                        mk(cold, lambda t: t, moe.BANK_HOST), rmd, H, I)
    b8 = LayerBuffers.allocate(T, k, H, I, E - 4, 4, i8=True)
    outs = []
    for kw in ({}, {"cold_stream": torch.cuda.Stream()}, {"hot_stream": torch.cuda.Stream()}):
        b8.out.zero_()
        i8.forward(xd, ids, w, b8, **kw)
        torch.cuda.synchronize()
        outs.append(b8.out[:T].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    # against the product of the unquantised activations: each of x and h is off
    # by at most half a step of 1/127 of its row's maximum, about 0.6 % in norm
    # for these rows (sqrt(1/12) / 127 * max/rms, max/rms below 4), taken four times
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gu = (rows["w13"][e].double() * rows["s13"][e].double()[:, None]) @ x[t].double()
            h = layer_ref.swiglu(gu[:I], gu[I:])
            want[t] += float(w[t, j]) * (rows["w2"][e].double() * rows["s2"][e].double()[:, None]) @ h
    got = outs[0].cpu().view(torch.bfloat16).double()
    assert float((got - want).norm() / want.norm()) <= 4 * 2 ** 0.5 * (1 / 12) ** 0.5 / 127 * 4


def test_every_scale_byte():
    """Scale bytes 1 .. 252 (products down to the subnormals, up to the type's
    range): the step's tokens see each byte in both products, the activations
    and weights scaled so that h and out stay finite."""
    T, k, H, I = 4, 1, 512, 512
    for lo, hi in ((1, 40), (100, 150), (215, 252)):
        E = 4
        rng = np.random.default_rng(lo)
        arr = {"hot": {"w13": rng.integers(0, 256, (E, 2 * I, H // 2), dtype=np.uint8),
                       "s13": rng.integers(lo, hi + 1, (E, 2 * I, H // 32)).astype(np.uint8),
                       "w2": rng.integers(0, 256, (E, H, I // 2), dtype=np.uint8),
                       "s2": np.full((E, H, I // 32), 100, np.uint8)}}
        arr["cold"] = {n: v[:0] for n, v in arr["hot"].items()}
        # gate and up of order one at most, whatever the bytes
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(lo))
        x = (x * 2.0 ** (127 - hi - 8)).to(torch.bfloat16) if hi > 127 else x.to(torch.bfloat16)
        ids = torch.arange(T, dtype=torch.int32)[:, None]
        w = torch.ones(T, 1)
        rm = np.arange(E)
        out, _ = run(arr, rm, ids, w, x, H, I)
        ref, bound, _ = layer_ref.layer(arr, row_of(rm, E, 0), x, ids, w, H, I)
        # tiny h flush nowhere, but bf16 itself ends at 2^-133: half of its last
        # step for h, times the down row, and for out
        w2 = torch.stack([layer_ref.mxfp4(arr["hot"]["w2"][e], arr["hot"]["s2"][e]).abs().sum(dim=1)
                          for e in range(E)])
        bound = bound + 2.0 ** -133 * w2 + 2.0 ** -133
        off = (out.double() - ref).abs()
        assert bool((off <= bound).all()), (lo, float((off / bound).max()))
