"""moe_topk_gate against the definition in 64 bits: ids exactly, weights within
the fp32 roundings of the softmax; ties, masked experts, strides and types."""
import math

import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def gate(logits, k, norm, stream=None):
    T = logits.shape[0]
    ids = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), 77.0, device="cuda")
    torch.cuda.synchronize()
    moe.moe_topk_gate(logits, ids[:T], w[:T], norm=norm, stream=stream)
    torch.cuda.synchronize()
    assert (ids[T] == 77).all() and (w[T] == 77).all()
    return ids[:T].cpu().numpy(), w[:T].cpu().double().numpy()


def reference(logits, k, norm):
    l = logits.double().cpu().numpy()
    T, E = l.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        there = [e for e in range(E) if l[t, e] > -math.inf]  # false for NaN too
        best = sorted(there, key=lambda e: (-l[t, e], e))[:k]
        if best:
            top = l[t, best[0]]
            ex = {e: 1.0 if l[t, e] == top else math.exp(l[t, e] - top) for e in there}
            total = sum(ex[e] for e in (best if norm == moe.GATE_NORM_PICKS else there))
            ids[t, :len(best)] = best
            w[t, :len(best)] = [ex[e] / total for e in best]
    return ids, w


def check(logits, k, norm):
    ids, w = gate(logits, k, norm)
    rid, rw = reference(logits, k, norm)
    assert np.array_equal(ids, rid)
    # l - max rounds by 2^-24 |l - max|, which the exponential turns into a
    # relative error of that size; exp, the sum of E terms and the quotient add
    # (E + 8) * 2^-24
    l = logits.double().cpu().numpy()
    spread = np.where(np.isfinite(l), np.abs(l), 0).max() * 2
    tol = (logits.shape[1] + 8 + 2 * spread) * 2.0 ** -24
    assert (np.abs(w - rw) <= tol * rw + 2.0 ** -126).all()


CASES = [(1, 1, 1), (1, 8, 8), (7, 384, 6), (5, 63, 3), (64, 65, 32), (130, 128, 2),
         (33, 257, 8), (3, 4096, 32), (9, 1025, 5), (4097, 16, 1), (2, 512, 7), (6, 300, 6)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_against_64_bits(T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 7 + E)
    l = (torch.randn(T, E, generator=g) * 3).to(dtype).cuda()
    for norm in (moe.GATE_NORM_PICKS, moe.GATE_NORM_ALL):
        check(l, k, norm)


def test_ties_zeros_and_strides():
    wide = torch.full((9, 101), 1e30, device="cuda")
    l = wide[:, 1:98]  # rows 4 bytes off a 16-byte boundary, 101 apart
    l.copy_(torch.randint(-2, 3, (9, 97), generator=torch.Generator().manual_seed(1)).float())
    l[0] = 0.0
    l[0, ::2] = -0.0     # the two zeros are equal: ascending ids
    l[1] = -7.25
    for norm in (moe.GATE_NORM_PICKS, moe.GATE_NORM_ALL):
        check(l, 8, norm)
    ids, _ = gate(l, 8, moe.GATE_NORM_PICKS)
    assert list(ids[0]) == list(ids[1]) == list(range(8))


def test_masked_rows():
    l = torch.randn(6, 70, generator=torch.Generator().manual_seed(2))
    l[0] = -math.inf                    # nothing left
    l[1] = math.nan
    l[2, 3:] = -math.inf                # fewer left than picks
    l[3, :35] = math.nan
    l[4] = torch.finfo(torch.float32).min  # the type's lowest value is not a mask
    l[5, 69] = -3e38
    l = l.cuda()
    for norm in (moe.GATE_NORM_PICKS, moe.GATE_NORM_ALL):
        check(l, 5, norm)
    ids, w = gate(l, 5, moe.GATE_NORM_PICKS)
    assert (ids[:2] == -1).all() and (w[:2] == 0).all() and (ids[2, 3:] == -1).all()
    assert list(ids[4]) == [0, 1, 2, 3, 4] and np.allclose(w[4], 0.2)


def test_infinite_logits_share_the_weight():
    l = torch.zeros(1, 40, device="cuda")
    l[0, 7] = l[0, 30] = math.inf
    for norm in (moe.GATE_NORM_PICKS, moe.GATE_NORM_ALL):
        ids, w = gate(l, 3, norm)
        assert list(ids[0]) == [7, 30, 0] and list(w[0]) == [0.5, 0.5, 0.0]


def test_offsets_past_32_bits():
    """Rows 2^30 elements apart: the third starts 4 GB into the buffer."""
    flat = torch.zeros(2 * 2 ** 30 + 64, dtype=torch.bfloat16, device="cuda")
    l = flat.as_strided((3, 64), (2 ** 30, 1))
    l.copy_(torch.randn(3, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16))
    check(l, 6, moe.GATE_NORM_ALL)


def test_feeds_the_split_and_the_layer():
    """Gate, then the split path and the few-token layer on its output, against
    the 64-bit layer; one token has every expert masked."""
    import layer_ref
    import synth
    from gpu_util import REL_L2, device_bank, host_bank, pinned_bank
    T, k, E, H, I = 6, 3, 10, 256, 192
    rm, ho, co = synth.random_map(E, 4, 3)
    arr = {n: host_bank(o, 3, 0, H, I, scale_lo=118, scale_cnt=4)
           for n, o in (("hot", ho), ("cold", co))}
    x = torch.from_numpy(synth.activations(T, H, 3).view(np.int16)).view(torch.bfloat16)
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(5))
    l[2] = -math.inf
    hot, cold = device_bank(arr["hot"]), pinned_bank(arr["cold"])
    rmd = torch.from_numpy(rm.astype(np.int32)).cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_layer_few_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    moe.moe_topk_gate(l.cuda(), ids, w)
    moe.moe_layer_few_mxfp4(hot, cold, rmd, x.cuda(), ids, w, I, ws, out, ninv)
    torch.cuda.synchronize()

    def row(e):
        return None if e < 0 else (("hot", int(rm[e])) if rm[e] >= 0 else ("cold", -1 - int(rm[e])))
    ref, bound, bad = layer_ref.layer(arr, row, x, ids.cpu(), w.cpu(), H, I)
    off = (out.cpu().double() - ref).abs()
    assert int(ninv) == bad == k and bool((off <= bound).all())
    assert float(off.norm() / ref.norm()) <= REL_L2 and (out[2] == 0).all()


def test_graph_replays():
    T, E, k = 40, 200, 4
    st = torch.zeros(T, E, device="cuda")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.moe_topk_gate(st, ids, w)
    for s in range(4):
        l = torch.randn(T, E, generator=torch.Generator().manual_seed(s)).cuda()
        st.copy_(l)
        g.replay()
        torch.cuda.synchronize()
        wi, ww = gate(l, k, moe.GATE_NORM_PICKS)
        assert np.array_equal(ids.cpu().numpy(), wi) and np.array_equal(w.cpu().double().numpy(), ww)


def masked_step(T, E, k, seed):
    """Logits with every kind of masked row among ordinary ones."""
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(seed))
    l[0] = -math.inf               # no expert left
    l[1, 1:] = math.nan            # one
    l[T - 2, k - 1:] = -math.inf   # one fewer than the picks
    return l


STALE = [0, 0x7fc1, 0xff80, 0x4228]  # +0, NaN, -inf, 42 (bf16 bits)


@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("kind", ["mxfp4", "i8"])
def test_masked_picks_add_nothing_on_the_split_path(kind, T):
    """Gate -> split -> expert FFN -> finalize where tokens have fewer unmasked
    experts than picks: the rows of Y that no bank writes hold what earlier steps
    left, and the output does not depend on it."""
    import layer_ref
    import synth
    from expert_weight_residency_amd.layer import LayerBuffers, ResidencyLayer
    from gpu_util import device_bank, host_bank, pinned_bank
    k, E, H, I = 3, 10, 256, 192
    rm, ho, co = synth.random_map(E, 4, 3)
    if kind == "mxfp4":
        arr = {n: host_bank(o, 3, 0, H, I, scale_lo=118, scale_cnt=4)
               for n, o in (("hot", ho), ("cold", co))}
        hot, cold = device_bank(arr["hot"]), pinned_bank(arr["cold"])
    else:
        def bank(rows):
            return moe.BankI8(torch.randint(-127, 128, (rows, 2 * I, H), dtype=torch.int8, generator=g).cuda(),
                              torch.full((rows, 2 * I), 1 / (73 * H ** 0.5), device="cuda"),
                              torch.randint(-127, 128, (rows, H, I), dtype=torch.int8, generator=g).cuda(),
                              torch.full((rows, H), 1 / (73 * I ** 0.5), device="cuda"))
        g = torch.Generator().manual_seed(4)
        hot, cold = bank(E - 4), bank(4)
    x = torch.from_numpy(synth.activations(T, H, 3).view(np.int16)).view(torch.bfloat16)
    l = masked_step(T, E, k, 5)
    layer = ResidencyLayer(hot, cold, torch.from_numpy(rm.astype(np.int32)).cuda(), H, I)
    bufs = LayerBuffers.allocate(T, k, H, I, E - 4, 4, i8=kind == "i8")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    layer.route(l.cuda(), ids, w)
    want = None
    for bits in STALE:
        bufs.Y.fill_(bits if bits < 0x8000 else bits - 0x10000)
        bufs.out.fill_(7)
        layer.forward(x.cuda(), ids, w, bufs)
        torch.cuda.synchronize()
        out = bufs.out[:T].cpu()
        want = out if want is None else want
        assert torch.equal(out, want), hex(bits)
        assert int(bufs.n_invalid) == int((ids < 0).sum()) == k + (k - 1) + 1
    got = want.view(torch.bfloat16).double()
    assert (got[0] == 0).all() and got.isfinite().all() and (got[1] != 0).any()
    if kind == "mxfp4" and T < 256:
        def row(e):
            return None if e < 0 else (("hot", int(rm[e])) if rm[e] >= 0 else ("cold", -1 - int(rm[e])))
        ref, bound, _ = layer_ref.layer(arr, row, x, ids.cpu(), w.cpu(), H, I)
        # besides the roundings of the bound, each row of Y to bf16: at most
        # 2^-8 of the row, whose weighted sum over the picks is at most that of
        # the weights times the largest row
        rows = bufs.Y[:T * k].cpu().view(torch.bfloat16).double().view(T, k, H).abs()
        rows = torch.where(ids.cpu()[:, :, None] < 0, 0.0, rows)
        extra = layer_ref.UBF16 * (1 + layer_ref.UBF16) * (w.cpu().double()[:, :, None] * rows).sum(dim=1)
        assert bool(((got - ref).abs() <= bound + extra).all())


def test_finalize_leaves_out_picks_of_weight_zero():
    """Bit for bit the chain over the finite rows; rows of infinities and NaN
    count where their weight is not 0, and only there."""
    import oracle
    T, k, H = 9, 5, 264
    rng = np.random.default_rng(6)
    Y = oracle.f32_to_bf16(rng.standard_normal((T * k, H)).astype(np.float32))
    w = rng.random((T, k)).astype(np.float32)
    special = np.array([0x7f80, 0xff80, 0x7fc0, 0xffff, 0x7f81, 0x8000], np.uint16)
    for t in range(1, 7):
        w[t, t % k] = 0.0 if t % 2 else -0.0
        Y[t * k + t % k] = rng.choice(special, H)
    w[7, 2] = 0.0                              # a finite row of weight 0
    Y[8 * k + 1, ::3] = 0x7fc0                 # NaN that counts
    out = torch.empty(T, H, dtype=torch.int16, device="cuda")
    moe.moe_finalize(torch.from_numpy(Y.view(np.int16)).cuda(), torch.from_numpy(w).cuda(), out)
    torch.cuda.synchronize()
    got = out.cpu().numpy().view(np.uint16)
    clean = Y.copy()
    for t in range(1, 7):
        row = clean[t * k + t % k]
        row[(row & 0x7f80) == 0x7f80] = 0
    want = oracle.finalize(clean.reshape(T, k, H), w)
    assert np.array_equal(got[:8], want[:8])
    nan = oracle.bf16_to_f32(got[8])
    assert np.isnan(nan[::3]).all() and np.isfinite(nan[1::3]).all()
    assert np.array_equal(got[8][1::3], want[8][1::3])
