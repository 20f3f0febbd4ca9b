"""Every scale byte through both products of the few-token layer, with the
experts in device and in pinned host memory."""
import numpy as np
import pytest
import torch

import expert_weight_residency_amd as moe
import layer_ref
from test_gpu_layer_few import row_of, run

pytestmark = pytest.mark.gpu

T = E = 2  # a token for each expert


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.lib()
    yield


def rows_of_byte(shape, byte, rng):
    """Weight rows whose scale of interest is `byte`: two blocks of each row have
    it, at places of their own; the other blocks hold zero codes under any other
    byte but NaN's, so that what stands beside a scale byte varies and adds
    nothing."""
    n, rows, cols = shape
    blocks = cols // 32
    scales = rng.integers(0, 255, (n, rows, blocks)).astype(np.uint8)
    codes = np.zeros((n, rows, blocks, 16), np.uint8)
    at = np.argsort(rng.random((n, rows, blocks)), axis=2)[:, :, :2]
    np.put_along_axis(scales, at, byte, axis=2)
    # 4 and 6 times 2^126 and 2 times 2^127 are past bf16's range: magnitudes up to 1.5 there
    some = np.array([0, 1, 2, 3, 8, 9, 10, 11] if byte >= 253 else range(16), np.uint8)
    pick = rng.choice(some, (n, rows, 2, 16)) | rng.choice(some, (n, rows, 2, 16)) << 4
    np.put_along_axis(codes, at[..., None], pick, axis=2)
    return codes.reshape(n, rows, cols // 2), scales


def largest_h(w13, s13, x, w, I):
    """Each token's largest |w h|, which the layer holds in fp32 and then bf16."""
    most = torch.zeros(E, dtype=torch.float64)
    for e in range(E):
        gu = layer_ref.mxfp4(w13[e], s13[e]) @ x[e].double()
        most[e] = (w[e].double() * layer_ref.swiglu(gu[:I], gu[I:])).abs().max()
    return most


@pytest.mark.parametrize("first", range(0, 255, 15))
@pytest.mark.parametrize("H,I", [(576, 1088), (4096, 192)])
def test_every_scale_byte(H, I, first):
    pairs = [(b, (37 * b + 11) % 255) for b in range(first, first + 15)]  # every byte once in both products
    while pairs:
        b, c = pairs.pop(0)
        rng = np.random.default_rng(b)
        w13, s13 = rows_of_byte((E, 2 * I, H), b, rng)
        w2, s2 = rows_of_byte((E, H, I), c, rng)
        hot = {"w13": w13, "s13": s13, "w2": w2, "s2": s2}
        arr = {"hot": hot, "cold": {n: v[:0] for n, v in hot.items()}}
        # gate and up around one, and out inside bf16's range, for most bytes
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(b))
        x = (x * 2.0 ** float(np.clip(124 - b, -110, 110))).to(torch.bfloat16)
        w = torch.full((T, 1), 2.0 ** float(np.clip(123 - c, -100, 100)))
        ids = torch.arange(E, dtype=torch.int32)[:, None]
        rm = np.arange(E)
        out, _ = run(arr, rm, ids, w, x, H, I)
        host, _ = run(arr, rm, ids, w, x, H, I, ("host", "device"))
        over = largest_h(w13, s13, x, w, I) >= 2.0 ** 128
        if over.any():
            # the weighted h, which the definition rounds to bf16, is past that
            # type (b = 248, c = 7: g and u reach 2^17, w is 2^100): no finite
            # result; the first product's byte runs beside another
            assert not out[over].isfinite().any() and not host[over].isfinite().any(), (b, c)
            pairs.append((b, 120))
            continue
        ref, bound, _ = layer_ref.layer(arr, row_of(rm, E, 0), x, ids, w, H, I)
        # bf16 ends at steps of 2^-133: half of one for the weighted h, times the
        # down row, and for out
        rows = torch.stack([layer_ref.mxfp4(w2[e], s2[e]).abs().sum(dim=1) for e in range(E)])
        bound = bound + 2.0 ** -134 * rows + 2.0 ** -134
        off = (out.double() - ref).abs()
        assert bool((off <= bound).all()), (b, c, float((off / bound).max()))
        # the bound is tight enough to tell one byte from the next
        assert float((ref.abs() > 4 * bound).double().mean()) > 0.7, (b, c)
        assert torch.equal(host.view(torch.int16), out.view(torch.int16)), (b, c)
    assert {b for b in range(255)} == {(37 * b + 11) % 255 for b in range(255)}
