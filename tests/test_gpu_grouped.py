"""The products grouped by expert and their gradients against their 64-bit forms, each
output within its fp32 sum's and its own type's rounding: ragged groups from no row to
thousands, odd sizes, both types, rows per token and per slot, banks, streams, graphs,
and a routed layer of them with its gradients against autograd and differences."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import synth
from layer_ref import HALF_STEP, U32

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def make_split(ids, E, rm=None, n_cold=0):
    T, k = ids.shape
    rm = np.arange(E) if rm is None else rm
    hot, cold = moe.Split.empty(E - n_cold, T, k), moe.Split.empty(n_cold, T, k)
    moe.moe_route_split(ids.cuda(), torch.from_numpy(np.ascontiguousarray(rm, np.int32)).cuda(), E - n_cold,
                        n_cold, hot, cold, torch.zeros(1, dtype=torch.int32, device="cuda"))
    return hot, cold


def inputs(T, k, E, N, K, dtype, by_token, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T if by_token else T * k, K, generator=g).to(dtype)
    dy = torch.randn(T * k, N, generator=g).to(dtype)
    w = (torch.randn(E, N, K, generator=g) / K ** 0.5).to(dtype)
    return x, dy, w


def routing(T, k, E):
    if k > E:  # ids repeat within a token
        return torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(T))
    return torch.from_numpy(synth.gaussian_routing(T, k, E, 5)[0].astype(np.int32))


def slots_of(ids, e):
    return (ids.reshape(-1) == e).nonzero().squeeze(1)


def close(got, ref, size, n, what):
    """got within an fp32 sum of n products of total magnitude size, and its rounding."""
    off = 2 * n * U32 * size
    tol = off + HALF_STEP[got.dtype] * (ref.abs() + off) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -140)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, float((err / tol).max()))


def run(x, dy, w, split, k, out, grad, stream=None):
    T_k, (E, N, K) = dy.shape[0], w.shape
    y = torch.full((T_k + 1, N), 7.0, dtype=out, device="cuda")
    dx = torch.full((T_k + 1, K), 7.0, dtype=out, device="cuda")
    dw = torch.full((E + 1, N, K), 7.0, dtype=grad, device="cuda")
    torch.cuda.synchronize()
    moe.moe_grouped_linear(x, w, split, k, y[:T_k], stream=stream)
    moe.moe_grouped_linear_dx(dy, w, split, k, dx[:T_k], stream=stream)
    moe.moe_grouped_linear_dw(dy, x, split, k, dw[:E], stream=stream)
    torch.cuda.synchronize()
    assert (y[T_k] == 7.0).all() and (dx[T_k] == 7.0).all() and (dw[E] == 7.0).all()
    return y[:T_k], dx[:T_k], dw[:E]


def check(ids, x, dy, w, y, dx, dw, experts=None):
    T, k = ids.shape
    E, N, K = w.shape
    per = k if x.shape[0] == T else 1
    left = torch.ones(T * k, dtype=torch.bool)
    for e in range(E) if experts is None else experts:
        s = slots_of(ids, e)
        left[s] = False
        xe, dye, we = x[s // per].double(), dy[s].double(), w[e].double()
        close(y[s.cuda()], xe @ we.T, xe.abs() @ we.abs().T, K, ("y", e))
        close(dx[s.cuda()], dye @ we, dye.abs() @ we.abs(), N, ("dx", e))
        close(dw[e], dye.T @ xe, dye.abs().T @ xe.abs(), len(s), ("dw", e))
    if experts is None:  # rows of no expert stay as they were
        assert (y[left.cuda()] == 7.0).all() and (dx[left.cuda()] == 7.0).all()


CASES = [
    # T, k, E, N, K
    (1, 1, 1, 8, 8),
    (1, 2, 4, 24, 40),
    (1, 6, 40, 256, 1440),
    (7, 6, 12, 576, 1024),
    (16, 3, 4, 4096, 2880),
    (5, 2, 6, 320, 8192),
    (3, 2, 3, 8256, 72),
    (40, 4, 64, 832, 192),
    (65, 1, 1, 136, 64),       # one row past a tile
    (130, 6, 16, 200, 264),    # part-filled tiles
    (700, 2, 3, 320, 128),     # several tiles per expert
    (257, 3, 2, 136, 1000),
    (64, 32, 40, 64, 64),
    (4, 3, 4096, 8, 16),
    (1500, 4, 5, 16, 2048),    # low rank
    (900, 2, 7, 2048, 16),
    (2500, 4, 4, 520, 648),    # experts of thousands of rows
]


@pytest.mark.parametrize("T,k,E,N,K", CASES)
@pytest.mark.parametrize("dtype", TYPES)
def test_products(T, k, E, N, K, dtype):
    ids = routing(T, k, E)
    split, _ = make_split(ids, E)
    for by_token, out, grad in ((True, dtype, torch.float32), (False, torch.float32, dtype)):
        x, dy, w = inputs(T, k, E, N, K, dtype, by_token, T + E)
        y, dx, dw = run(x.cuda(), dy.cuda(), w.cuda(), split, k, out, grad)
        few = None if E * N * K < 2 ** 27 else torch.unique(ids).tolist()[:6]
        check(ids, x, dy, w, y, dx, dw, few)


@pytest.mark.parametrize("T,E", [(300, 9), (4, 4096)])
def test_other_output_types(T, E):
    """Inputs of one 16-bit type, outputs of the other."""
    k, N, K = 2, 40, 72
    ids, _ = synth.gaussian_routing(T, k, E, 6)
    ids = torch.from_numpy(ids.astype(np.int32))
    split, _ = make_split(ids, E)
    for dtype, other in (TYPES, TYPES[::-1]):
        x, dy, w = inputs(T, k, E, N, K, dtype, True, 3)
        check(ids, x, dy, w, *run(x.cuda(), dy.cuda(), w.cuda(), split, k, other, other))


@pytest.mark.parametrize("T", [6, 300])
def test_invalid_picks_and_empty_experts(T):
    """Picks of no expert leave their rows as they were, whatever those hold; experts
    without a row get zero gradients."""
    k, E, N, K = 3, 70, 72, 136
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, 5, (T, k), dtype=torch.int32, generator=g) * 13  # 0, 13, .. 52: most stay empty
    ids[0, 1], ids[T - 1], ids[2, 0] = -1, E + 3, 69
    ids[:, 2] = ids[:, 0]                                                   # an id twice
    split, _ = make_split(ids, E)
    for by_token in (True, False):
        x, dy, w = inputs(T, k, E, N, K, torch.bfloat16, by_token, 1)
        gone = (ids.reshape(-1) < 0) | (ids.reshape(-1) >= E)
        dy[gone] = float("nan")
        if not by_token:
            x[gone] = float("inf")
        unused = [e for e in range(E) if not (ids == e).any()]
        w[unused] = float("nan")
        y, dx, dw = run(x.cuda(), dy.cuda(), w.cuda(), split, k, torch.bfloat16, torch.float32)
        w[unused] = 0
        check(ids, x, dy, w, y, dx, dw)
        assert (dw[unused] == 0).all() and dw.isfinite().all()


def test_special_values_stay_in_their_rows():
    T, k, E, N, K = 90, 2, 3, 72, 200
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=g)
    split, _ = make_split(ids, E)
    x, dy, w = inputs(T, k, E, N, K, torch.float16, False, 2)
    base = run(x.cuda(), dy.cuda(), w.cuda(), split, k, torch.float32, torch.float32)
    x2, dy2 = x.clone(), dy.clone()
    x2[7, 3], dy2[11, 5] = float("nan"), float("inf")
    y, dx, dw = run(x2.cuda(), dy2.cuda(), w.cuda(), split, k, torch.float32, torch.float32)
    rest = [s for s in range(T * k) if s not in (7, 11)]
    assert y[7].isnan().all() and not dx[11].isfinite().any()
    assert torch.equal(y[rest], base[0][rest]) and torch.equal(dx[rest], base[1][rest])
    e7, e11 = int(ids.reshape(-1)[7]), int(ids.reshape(-1)[11])
    assert dw[e7][:, 3].isnan().all() and not dw[e11][5].isfinite().any()
    clean = torch.ones(E, N, K, dtype=torch.bool)
    clean[e7][:, 3], clean[e11][5] = False, False
    assert torch.equal(dw[clean.cuda()], base[2][clean.cuda()])


def test_no_valid_picks_and_no_tokens():
    k, E, N, K = 2, 5, 16, 24
    ids = torch.full((9, k), -1, dtype=torch.int32)
    split, _ = make_split(ids, E)
    x, dy, w = inputs(9, k, E, N, K, torch.bfloat16, True, 1)
    y, dx, dw = run(x.cuda(), dy.cuda(), w.cuda(), split, k, torch.bfloat16, torch.float32)
    assert (y == 7.0).all() and (dx == 7.0).all() and (dw == 0).all()
    stale, _ = make_split(torch.zeros(9, k, dtype=torch.int32), E)  # a split of an earlier, larger step
    none = torch.empty(0, K, dtype=torch.bfloat16, device="cuda"), torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    y, dx, dw = run(none[0], none[1], w.cuda(), stale, k, torch.bfloat16, torch.bfloat16)
    assert (dw == 0).all()


def test_banks_and_streams():
    """Hot experts in HBM and cold ones in pinned memory, on two streams: the bits of
    one bank."""
    T, k, E, n_cold, N, K = 50, 4, 12, 5, 320, 520
    ids, _ = synth.gaussian_routing(T, k, E, 7)
    ids = torch.from_numpy(ids.astype(np.int32))
    x, dy, w = inputs(T, k, E, N, K, torch.bfloat16, True, 9)
    one, _ = make_split(ids, E)
    want = run(x.cuda(), dy.cuda(), w.cuda(), one, k, torch.bfloat16, torch.bfloat16)
    rm, ho, co = synth.random_map(E, n_cold, 4)
    hot, cold = make_split(ids, E, rm, n_cold)
    xd, dyd = x.cuda(), dy.cuda()
    wh, wc = w[torch.as_tensor(ho).long()].cuda(), w[torch.as_tensor(co).long()].pin_memory()
    y = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(T * k, K, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        y.fill_(0), dx.fill_(0)
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_grouped_linear(xd, wc, cold, k, y, stream=side)
        moe.moe_grouped_linear_dx(dyd, wc, cold, k, dx, stream=side)
        moe.moe_grouped_linear(xd, wh, hot, k, y)
        moe.moe_grouped_linear_dx(dyd, wh, hot, k, dx)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
    for split, owners in ((hot, ho), (cold, co)):
        dw = torch.empty(len(owners), N, K, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_linear_dw(dyd, xd, split, k, dw)
        torch.cuda.synchronize()
        assert torch.equal(dw, want[2][torch.as_tensor(owners).long().cuda()])


@pytest.mark.parametrize("T", [8, 400])
def test_graph_replays_match_eager(T):
    k, E, N, K = 4, 16, 200, 328
    steps = []
    for s in range(4):
        ids, _ = synth.gaussian_routing(T, k, E, 30 + s)
        ids = torch.from_numpy(ids.astype(np.int32))
        ids[s] = -1
        x, dy, w = inputs(T, k, E, N, K, torch.bfloat16, True, s)
        steps.append([ids.cuda(), x.cuda(), dy.cuda(), w.cuda()])
    st = [t.clone() for t in steps[0]]
    split, none = moe.Split.empty(E, T, k), moe.Split.empty(0, T, k)
    rm = torch.arange(E, dtype=torch.int32, device="cuda")
    ninv = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda"),
            torch.zeros(T * k, K, dtype=torch.float32, device="cuda"),
            torch.zeros(E, N, K, dtype=torch.float32, device="cuda")]

    def step():
        moe.moe_route_split(st[0], rm, E, 0, split, none, ninv)
        moe.moe_grouped_linear(st[1], st[3], split, k, outs[0])
        moe.moe_grouped_linear_dx(st[2], st[3], split, k, outs[1])
        moe.moe_grouped_linear_dw(st[2], st[1], split, k, outs[2])

    def load(n):
        for d, v in zip(st, steps[n]):
            d.copy_(v)
        for o in outs:
            o.fill_(3)

    want = []
    for n in range(4):
        load(n)
        step()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for rep in range(6):
        n = (rep * 3) % 4
        load(n)
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want[n]):
            assert torch.equal(got, ref)
        assert torch.randn(64, 64, device="cuda").sum().isfinite()


def layer_step(x, w13, w2, ids, topk_w, split, k, dout):
    """A routed layer of unquantised experts with its gradients, the products from the
    library: gate/up, SwiGLU, down, the weighted sum; then back."""
    T, H = x.shape
    E, I2, _ = w13.shape
    I, S = I2 // 2, T * k
    t = x.dtype
    gu = torch.zeros(S, I2, device="cuda")
    moe.moe_grouped_linear(x, w13, split, k, gu)
    g, u = gu[:, :I], gu[:, I:]
    sig = torch.sigmoid(g)
    h = (g * sig * u).to(t)
    y = torch.zeros(S, H, dtype=t, device="cuda")
    moe.moe_grouped_linear(h, w2, split, k, y)
    out = torch.empty(T, H, dtype=t, device="cuda")
    moe.moe_finalize(y, topk_w, out)
    dy = (dout.float().repeat_interleave(k, 0) * topk_w.reshape(-1, 1)).to(t)
    dh = torch.zeros(S, I, device="cuda")
    moe.moe_grouped_linear_dx(dy, w2, split, k, dh)
    dw2 = torch.empty(E, H, I, device="cuda")
    moe.moe_grouped_linear_dw(dy, h, split, k, dw2)
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=1).to(t)
    dxs = torch.zeros(S, H, dtype=t, device="cuda")
    moe.moe_grouped_linear_dx(dgu, w13, split, k, dxs)
    dw13 = torch.empty(E, I2, H, device="cuda")
    moe.moe_grouped_linear_dw(dgu, x, split, k, dw13)
    dx = torch.empty(T, H, dtype=t, device="cuda")
    moe.moe_finalize(dxs, torch.ones_like(topk_w), dx)
    return out, dx, dw13, dw2


def test_a_routed_layer_and_its_gradients():
    """Gate, split, the products, their gradients together, against 64-bit autograd and
    against differences of the 64-bit loss. Relative L2 errors: every value passes at
    most 5 roundings to bf16 (h, y or dy, dgu, the slots' rows, the output), each at
    most 2^-8 of it, whose errors' signs the products average."""
    T, k, E, H, I = 48, 3, 6, 128, 192
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(T, E, generator=g)
    x = torch.randn(T, H, generator=g).bfloat16()
    w13 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).bfloat16()
    w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).bfloat16()
    dout = torch.randn(T, H, generator=g).bfloat16()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, k, device="cuda")
    moe.moe_topk_gate(logits.cuda(), ids, tw)
    split, _ = make_split(ids.cpu(), E)
    got = layer_step(x.cuda(), w13.cuda(), w2.cuda(), ids, tw, split, k, dout.cuda())
    torch.cuda.synchronize()
    leaves = [v.double().requires_grad_() for v in (x, w13, w2)]

    def loss(x, w13, w2):
        gu = torch.einsum("tkih,th->tki", w13[ids.cpu().long()], x)
        h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
        y = torch.einsum("tkhi,tki->tkh", w2[ids.cpu().long()], h)
        out = (y * tw.cpu().double().unsqueeze(2)).sum(1)
        return out, (out * dout.double()).sum()
    out, l = loss(*leaves)
    grads = torch.autograd.grad(l, leaves)
    for name, a, b in zip(("out", "dx", "dw13", "dw2"), got, (out.detach(), *grads)):
        a = a.cpu().double()
        assert float((a - b).norm() / b.norm()) <= 5 * 2.0 ** -8, name
    # a difference of the loss along a direction is the gradients' product with it
    way = [torch.randn(v.shape, generator=g, dtype=torch.float64) for v in leaves]
    eps = 1e-6
    with torch.no_grad():
        up = loss(*[v + eps * d for v, d in zip(leaves, way)])[1]
        dn = loss(*[v - eps * d for v, d in zip(leaves, way)])[1]
    slope = float((up - dn) / (2 * eps))
    mine = sum(float((a.cpu().double() * d).sum()) for a, d in zip(got[1:], way))
    size = sum(float(b.norm()) for b in grads)  # a random direction sees a gradient's norm
    assert abs(mine - slope) <= 4 * 5 * 2.0 ** -8 * size


def test_offsets_past_32_bits():
    """Weights and gradients of more than 4 GB, and rows of more than 4 GB."""
    T, k, E, N, K = 30, 2, 40, 8192, 8200
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(E, N, K, dtype=torch.bfloat16, device="cuda", generator=g)
    ids = torch.randint(E - 3, E, (T, k), dtype=torch.int32)
    split, _ = make_split(ids, E)
    x, dy, _ = inputs(T, k, 1, N, K, torch.bfloat16, True, 2)
    y, dx, dw = run(x.cuda(), dy.cuda(), w, split, k, torch.bfloat16, torch.bfloat16)
    last = w[E - 3:].cpu()
    for e in range(3):
        s = slots_of(ids, E - 3 + e)
        xe, dye, we = x[s // k].double(), dy[s].double(), last[e].double()
        close(y[s.cuda()], xe @ we.T, xe.abs() @ we.abs().T, K, "y")
        close(dx[s.cuda()], dye @ we, dye.abs() @ we.abs(), N, "dx")
        close(dw[E - 3 + e], dye.T @ xe, dye.abs().T @ xe.abs(), len(s), "dw")
    assert (dw[:E - 3] == 0).all()
    del w, y, dx, dw
    T, k, E, N, K = 300000, 1, 2, 16, 8192
    ids = torch.zeros(T, k, dtype=torch.int32)
    ids[T - 100:] = 1
    split, _ = make_split(ids, E)
    x = torch.randn(T, K, dtype=torch.bfloat16, device="cuda", generator=g)
    w = torch.randn(E, N, K, dtype=torch.bfloat16, device="cuda", generator=g)
    dy = torch.randn(T, N, dtype=torch.bfloat16, device="cuda", generator=g)
    y, dx, dw = run(x, dy, w, split, k, torch.bfloat16, torch.float32)
    for rows, e in ((slice(0, 5), 0), (slice(T - 101, T - 100), 0), (slice(T - 100, T), 1)):
        xe, dye, we = x[rows].cpu().double(), dy[rows].cpu().double(), w[e].cpu().double()
        close(y[rows], xe @ we.T, xe.abs() @ we.abs().T, K, "y")
        close(dx[rows], dye @ we, dye.abs() @ we.abs(), N, "dx")
    xe, dye = x[T - 100:].cpu().double(), dy[T - 100:].cpu().double()
    close(dw[1], dye.T @ xe, dye.abs().T @ xe.abs(), 100, "dw")
