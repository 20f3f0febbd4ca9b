"""Plain 64-bit forms of the 8-bit floating point products (torch on the CPU) and
elementwise bounds of what a kernel that rounds where the operator says may be
off by (the roundings as in layer_ref)."""
import torch

import layer_ref
from layer_ref import HALF_STEP, U32

BLOCK = 128
_code = torch.arange(256)
_field, _frac = (_code // 8) % 16, (_code % 8).double()
# E4M3 from its fields: sign, 4 bits of exponent (bias 7), 3 of fraction
VALUE = torch.where(_field == 0, _frac / 8 * 2.0 ** -6,
                    (1 + _frac / 8) * torch.exp2((_field - 7).double()))
VALUE = torch.where(_code >= 128, -VALUE, VALUE)
VALUE[[127, 255]] = float("nan")
GRID = VALUE[:127]  # 0 .. 448 in order


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def values(codes: torch.Tensor) -> torch.Tensor:
    return VALUE[codes.cpu().view(torch.uint8).long()]


def spread(scale: torch.Tensor, rows: int, cols: int, by_row: bool = False) -> torch.Tensor:
    """One scale per element from one per block (by_row: per row and block of columns)."""
    s = scale.double().repeat_interleave(BLOCK, -1)[..., :cols]
    return s if by_row else s.repeat_interleave(BLOCK, -2)[..., :rows, :]


def nearest(r: torch.Tensor) -> torch.Tensor:
    """The E4M3 value nearest to each r in [0, 448], the even code of two as near;
    r in 64 bits."""
    up = torch.searchsorted(GRID, r.contiguous()).clamp_max(126)
    down = (up - 1).clamp_min(0)
    over, under = GRID[up] - r, r - GRID[down]
    return GRID[torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)]


def quantize(x: torch.Tensor):
    """(values, magnitudes max|x| per element) of each row's blocks of 128."""
    x = x.double()
    rows, K = x.shape
    wide = torch.zeros(rows, blocks(K) * BLOCK, dtype=torch.float64)
    wide[:, :K] = x.abs()
    most = wide.view(rows, -1, BLOCK).amax(dim=2).repeat_interleave(BLOCK, 1)[:, :K]
    # 448 |x| is exact for 24-bit values; where the quotient lies half way between
    # two E4M3 values it is exact too, and no other rounds there in 64 bits
    q = nearest((x.abs() * 448 / torch.where(most > 0, most, 1.0)).clamp_max(448))
    return torch.sign(x) * q, most


# The FP8 matrix instruction, which products with 16-bit outputs use, cuts each of 8
# products at 2^-13 of the largest of them: 7 cuts of less than that.
CUT = 7 * 2.0 ** -13


def product(xv, xs, wv, ws, ydtype):
    """y in 64 bits and the bound of a kernel that sums a block's products in fp32
    (or as the FP8 instruction does, for a 16-bit output), multiplies by the two
    scales' product (one rounding) and adds blocks in fp32 by fma: sums of 128 and of
    the blocks by twice their half steps (layer_ref), one half step for the scales'
    product."""
    M, K = xv.shape
    s, w = spread(xs, M, K, True), spread(ws, wv.shape[0], K)
    y = (xv * s) @ (wv * w).T
    most = (xv * s).abs() @ (wv * w).abs().T
    cut = 0 if ydtype == torch.float32 else CUT
    return y, (cut + (2 * min(K, BLOCK) + 2 * blocks(K) + 2) * U32) * most


def ffn(x, bank, e, ydtype=torch.bfloat16):
    """Expert e's rows for the tokens x (any float type): y in 64 bits and its bound."""
    xq, xm = quantize(x)
    xs = xm / 448
    I = bank["w13"].shape[1] // 2
    full = {}
    for part, rows in (("g", slice(0, I)), ("u", slice(I, 2 * I))):
        w = values(bank["w13"][e, rows]) * spread(bank["s13"][e, 0 if part == "g" else 1], I, x.shape[1])
        v = (xq * xs) @ w.T
        # the fp32 scale of the activations is one rounding more than in product()
        off = (2 * BLOCK + 2 * blocks(x.shape[1]) + 3) * U32 * ((xq * xs).abs() @ w.abs().T)
        full[part] = (v, off)
    (g, dg), (u, du) = full["g"], full["u"]
    h, dh = layer_ref.swiglu(g, u), layer_ref.swiglu_bound(g, u, dg, du)
    hq, most = quantize(h)
    # the block's largest, and with it the step, is off by its own error at most
    wide = torch.zeros(h.shape[0], blocks(I) * BLOCK, dtype=torch.float64)
    wide[:, :I] = dh
    dm = wide.view(h.shape[0], -1, BLOCK).amax(dim=2).repeat_interleave(BLOCK, 1)[:, :I]
    safe = most.clamp_min(1e-300)
    rel = dm / safe
    r = (448 * h.abs() / safe).clamp_max(448)
    dr = 1.01 * (448 * dh / safe + r * rel)
    # a value may turn to its neighbour where r's error reaches past the middle
    low, high = nearest((r - dr).clamp_min(0)), nearest((r + dr).clamp_max(448))
    step = torch.maximum(high - hq.abs(), hq.abs() - low)
    w2 = values(bank["w2"][e]) * spread(bank["s2"][e], x.shape[1], I)
    s = most / 448
    y = (hq * s) @ w2.T
    size = ((hq.abs() + step) * s) @ w2.abs().T
    tol = (step * s) @ w2.abs().T + ((hq.abs() + step) * s * rel) @ w2.abs().T
    tol = tol + (CUT + (2 * BLOCK + 2 * blocks(I) + 4) * U32) * size
    return y, tol + HALF_STEP[ydtype] * (y.abs() + tol)
