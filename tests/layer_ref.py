"""Plain 64-bit forms of the operators around the residency split (torch on the
CPU, one pick or row at a time), and elementwise bounds of what a kernel that
rounds where the operator says may be off by.

A rounding to a type is off by at most eps/2 of the value (bf16 2^-8, fp16
2^-11, fp32 2^-24); a sum of n products in fp32 by at most n * 2^-24 of the sum
of their magnitudes, taken twice here since the matrix instructions' own
order and rounding are not specified further."""
import numpy as np
import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)
U32, UBF16, UF16 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
HALF_STEP = {torch.float32: U32, torch.bfloat16: UBF16, torch.float16: UF16}


def mxfp4(codes: np.ndarray, scales: np.ndarray) -> torch.Tensor:
    c, s = torch.from_numpy(codes).long(), torch.from_numpy(scales).double()
    v = E2M1[torch.stack((c & 15, c >> 4), dim=-1).flatten(-2)]
    two = torch.where(s == 255, float("nan"), torch.exp2(s - 127))
    return v * two.repeat_interleave(32, dim=-1)


def swiglu(g, u):
    return g * torch.sigmoid(g) * u


def swiglu_bound(g, u, dg, du):
    """|error| of fp32 silu(g) * u with g, u off by dg, du: |silu'| <= 1.1,
    |silu(g)| <= |g|; the exponential, quotient and products together within
    32 fp32 half steps."""
    return 1.1 * dg * u.abs() + g.abs() * du + dg * du + 32 * U32 * (g * u).abs()


def layer(banks: dict, row_of, x, ids, w, H: int, I: int):
    """out [T,H] in 64 bits of the routed MXFP4 layer, its elementwise bound for
    a kernel that rounds h (times the weight) and out to bf16, and the number
    of invalid picks. banks: name -> arrays; row_of(id) -> (name, row) or None."""
    T, k = ids.shape
    xd = x.double()
    out, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    invalid, deq = 0, {}
    for t in range(T):
        for j in range(k):
            at = row_of(int(ids[t, j]))
            if at is None:
                invalid += 1
                continue
            if at not in deq:
                b = banks[at[0]]
                deq[at] = (mxfp4(b["w13"][at[1]], b["s13"][at[1]]),
                           mxfp4(b["w2"][at[1]], b["s2"][at[1]]))
            w13, w2 = deq[at]
            gu = w13 @ xd[t]
            dgu = 2 * H * U32 * (w13.abs() @ xd[t].abs())
            g, u = gu[:I], gu[I:]
            h = swiglu(g, u)
            dh = swiglu_bound(g, u, dgu[:I], dgu[I:])
            wt = float(w[t, j])
            out[t] += wt * (w2 @ h)
            # h to bf16 (and the fp32 product with the weight), then sums over I and k
            off = UBF16 * (h.abs() + dh) + dh + 2 * U32 * h.abs()
            bound[t] += abs(wt) * (w2.abs() @ (off + 2 * (I + k) * U32 * (h.abs() + off)))
    return out, bound + UBF16 * (out.abs() + bound), invalid


def quantize(x: torch.Tensor):
    """The nearest of the 255 steps of each row's largest magnitude (ties to the
    even step) and the step, in 64 bits; x * 127 is exact for 24-bit values, a
    quotient half way between two steps is exact, and no other rounds there."""
    x = x.double()
    most = x.abs().amax(dim=1, keepdim=True)
    q = torch.round(x * 127 / torch.where(most > 0, most, 1.0))
    return q, most / 127
