"""nvfp4_matvec and mxfp4_matvec on terms whose sums are exact in every order: a
lost, doubled or misplaced term of a long row shows, where a tolerance that
grows with the row would cover it.

Activations are whole numbers, weights multiples of a unit (1/2 times the
smallest bit of a scale), and the terms' magnitudes add up to less than 2^24
units, so that every partial sum is an fp32 value: results equal the 64-bit
product (itself exact), bf16 ones its rounding.
"""
import pytest
import torch

from block_util import E2M1, E4M3

pytestmark = pytest.mark.gpu

BLOCK = {"nvfp4": 16, "mxfp4": 32}


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _weights64(q, s, fmt):
    """Bytes of some rows -> their values in float64."""
    e = torch.from_numpy(E2M1).to(q.device)[torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).long()]
    scale = torch.from_numpy(E4M3).to(q.device)[s.long()] if fmt == "nvfp4" else torch.exp2(s.double() - 127)
    return (e.unflatten(-1, (-1, BLOCK[fmt])) * scale[..., None]).flatten(-2)


def _check(nv, fmt, M, K, N, most, codes, unit):
    """x: whole numbers up to `most`; scales: `codes`, at which weights are multiples of `unit`."""
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(M + 3 * K + 5 * N)
    x = torch.randint(1, most + 1, (M, K), device="cuda:0", generator=gen)
    x = (x * (2 * torch.randint(0, 2, (M, K), device="cuda:0", generator=gen) - 1)).bfloat16()
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=gen)
    s = torch.randint(*codes, (N, K // BLOCK[fmt]), dtype=torch.uint8, device="cuda:0", generator=gen)
    gs = torch.tensor([0.5], device="cuda:0")
    got = {d: nv.matvec(x, q, s, gs, out_dtype=d) if fmt == "nvfp4" else nv.mx_matvec(x, q, s, out_dtype=d)
           for d in (torch.float32, torch.bfloat16)}
    xt = x.double().t().contiguous()
    step = max(1, 2 ** 25 // K)
    for n in range(0, N, step):
        w = _weights64(q[n:n + step], s[n:n + step], fmt)
        assert float((w.abs() @ xt.abs()).max()) < 2 ** 24 * unit
        ref = (w @ xt).t() * (0.5 if fmt == "nvfp4" else 1.0)
        assert torch.equal(got[torch.float32][:, n:n + step].double(), ref)
        assert torch.equal(got[torch.bfloat16][:, n:n + step], ref.float().bfloat16())


# E4M3 scales 1 to 3.75 with all their bits, E8M0 scales 1, 2 and 4
FULL = {"nvfp4": dict(most=3, codes=(0x38, 0x48), unit=1 / 16), "mxfp4": dict(most=3, codes=(127, 130), unit=1 / 2)}


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [2, 7, 13, 27, 45, 61])
@pytest.mark.parametrize("N", [77, 4200, 8300, 12400, 16384, 24700])
def test_matvec_every_kernel_over_long_rows(nv, fmt, M, N):
    """Each class of tokens with rows of W on every side of the bounds between
    the kernels and their tiles; K takes every one of them through its main loop,
    into a second (few tokens) or third (tiles) part of the scales, and ends
    inside a step and inside a chunk."""
    _check(nv, fmt, M, 18848, N, **FULL[fmt])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K,N", [(1, 17056, 40), (3, 33184, 33), (6, 32800, 66), (11, 32800, 5), (16, 17088, 20),
                                   (33, 24672, 9), (64, 8320, 50), (64, 8192, 18), (20, 16384, 35), (4, 16384, 20),
                                   (12, 32768, 16), (50, 16416, 40)])
def test_matvec_long_rows_at_the_parts_of_their_scales(nv, fmt, M, K, N):
    """Whole parts, and rests of one to four blocks behind them."""
    _check(nv, fmt, M, K, N, **FULL[fmt])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N", [(1, 3), (8, 17), (16, 5), (31, 2), (48, 33), (64, 2)])
def test_matvec_longest_rows(nv, fmt, M, N):
    codes = {"nvfp4": (0x38, 0x39), "mxfp4": (127, 129)}[fmt]  # 1; 1 and 2
    _check(nv, fmt, M, 2 ** 20, N, 1, codes, 1 / 2)
