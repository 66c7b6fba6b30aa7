"""GPU parity of nvfp4_matvec and mxfp4_matvec with a 64-bit product of the same bytes.

Tolerance: products are exact, so an fp32 result is off by the roundings of the
additions alone: at most (K + 2) 2^-24 times the sum of the terms' magnitudes
(every order of K additions, the tensor scale and the product with it), plus
half an fp32 step where results underflow.  bf16 results add half a bf16 step, 2^-8."""
import numpy as np
import pytest
import torch

from block_util import values, weights
from gpu_util import dev_bf16, host, host_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _run(nv, fmt, x, q, s, gs, dtype, **kw):
    if fmt == "nvfp4":
        return nv.matvec(x, q, s, gs, out_dtype=dtype, **kw)
    return nv.mx_matvec(x, q, s, out_dtype=dtype, **kw)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _gs(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda:0")


def _x_bits(rng, M, K):
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).bfloat16()
    return x.view(torch.int16).numpy().view(np.uint16), x.double().numpy()


def _check(got, ref, mag, K, dtype):
    got = got.double().cpu().numpy()
    tol = (K + 2) * 2.0 ** -24 * mag + 2.0 ** -149
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
    assert got.shape == ref.shape
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


SHAPES = [(1, 32, 1), (1, 1024, 512), (2, 64, 17), (3, 96, 15), (4, 7168, 100), (5, 1376, 257), (7, 160, 31),
          (8, 4096, 66), (9, 2080, 33), (12, 512, 1000), (16, 7168, 48), (17, 1376, 130), (31, 288, 16), (33, 1024, 65),
          (48, 480, 97), (64, 4096, 80), (65, 1024, 33), (130, 224, 70)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_matvec_against_64_bits(nv, fmt, M, K, N, dtype):
    rng = np.random.Generator(np.random.PCG64(M + 3 * K + 5 * N))
    bits, x = _x_bits(rng, M, K)
    q, s = weights(rng, N, K, fmt)
    g = np.float32(0.0123) if fmt == "nvfp4" else np.float32(1)
    w = values(q, s, fmt, g)
    y = _run(nv, fmt, dev_bf16(bits), _dev(q), _dev(s), _gs(g), dtype)
    _check(y, x @ w.T, np.abs(x) @ np.abs(w).T, K, dtype)


# sizes on both sides of every choice of a kernel: many rows, and rows longer
# than the scales that are staged at a time, with a rest behind whole steps
WIDE = [(1, 288, 12289), (3, 288, 16383), (2, 96, 16500), (4, 160, 28700), (6, 288, 12301), (8, 160, 16384),
        (7, 288, 16385), (8, 96, 24600), (9, 288, 8190), (12, 288, 8200), (16, 160, 16001), (13, 288, 16400),
        (20, 288, 4097), (30, 352, 8200), (47, 288, 8191), (40, 160, 8193), (64, 480, 5000), (64, 288, 8200),
        (50, 544, 16390), (100, 288, 2100), (130, 32, 6000),
        (1, 17056, 40), (3, 33184, 33), (8, 17056, 18), (6, 20000, 66), (16, 17088, 20), (11, 32800, 5),
        (20, 8352, 30), (40, 16800, 17), (64, 8320, 50), (33, 24672, 9), (1, 2 ** 20, 3), (64, 2 ** 20, 2),
        (40, 512, 4200), (20, 768, 9000), (64, 256, 8300), (16, 768, 12000), (64, 8192, 40), (64, 8704, 70), (33, 8960, 40),
        (14, 8448, 8300)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K,N", WIDE)
def test_matvec_many_and_long_rows(nv, fmt, M, K, N):
    rng = np.random.Generator(np.random.PCG64(M + 7 * K + N))
    bits, x = _x_bits(rng, M, K)
    q, s = weights(rng, N, K, fmt)
    g = np.float32(0.37) if fmt == "nvfp4" else np.float32(1)
    w = values(q, s, fmt, g)
    y = _run(nv, fmt, dev_bf16(bits), _dev(q), _dev(s), _gs(g), torch.float32)
    _check(y, x @ w.T, np.abs(x) @ np.abs(w).T, K, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K", [(10, 8480), (40, 8480), (12, 16544)])
def test_matvec_long_and_many_rows(nv, fmt, M, K):
    """The 64-row tiles with more than one part of the scales: a few rows of
    many against 64 bits, and every row against the same rows by themselves."""
    N = 16500
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(K + M)
    lo, hi, block = (0x20, 0x50, 16) if fmt == "nvfp4" else (118, 126, 32)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=gen)
    s = torch.randint(lo, hi, (N, K // block), dtype=torch.uint8, device="cuda:0", generator=gen)
    x = torch.randn(M, K, device="cuda:0", generator=gen).bfloat16()
    y = _run(nv, fmt, x, q, s, _gs(1.0), torch.float32)
    at = torch.tensor([0, 17, 63, 64, 8191, 16383, 16384, 16447, N - 1], device="cuda:0")
    w = values(q[at].cpu().numpy(), s[at].cpu().numpy(), fmt)
    xd = x.double().cpu().numpy()
    mag = np.abs(xd) @ np.abs(w).T
    _check(y[:, at], xd @ w.T, mag, K, torch.float32)
    for n in range(0, N, 4000):  # other kernels, other orders of the same sums
        part = _run(nv, fmt, x, q[n:n + 4000], s[n:n + 4000], _gs(1.0), torch.float32)
        assert float((part - y[:, n:n + 4000]).abs().max()) <= 4 * (K + 2) * 2.0 ** -24 * float(mag.max())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,K,N", [(1, 7168, 300), (4, 1376, 77), (6, 992, 130), (16, 2048, 65), (24, 4096, 48),
                                   (64, 1120, 35)])
def test_matvec_whole_numbers_are_exact(nv, fmt, M, K, N):
    """Terms that are multiples of 1/2 with sums below 2^23: every order of
    additions gives the sum itself, so a lost, doubled or misplaced term shows."""
    rng = np.random.Generator(np.random.PCG64(M * K + N))
    x = rng.integers(-8, 9, (M, K)).astype(np.float32)
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if fmt == "nvfp4":
        s = rng.integers(0x38, 0x60, (N, K // 16), dtype=np.uint8)  # 1 .. 30 in eighths: all bits of the scale
    else:
        s = rng.integers(127, 131, (N, K // 32), dtype=np.uint8)
    ref = x.astype(np.float64) @ values(q, s, fmt).T
    assert np.abs(ref).max() < 2 ** 20 and (np.abs(x) @ np.abs(values(q, s, fmt)).T).max() * 16 < 2 ** 27
    small = (np.abs(x) @ np.abs(values(q, s, fmt)).T) * 16 < 2 ** 24  # in units of 1/16
    y = _run(nv, fmt, torch.from_numpy(x).bfloat16().to("cuda:0"), _dev(q), _dev(s), _gs(1.0), torch.float32)
    got = host(y)
    assert small.mean() > 0.5 or K > 4000
    assert np.array_equal(got[small], ref[small].astype(np.float32))


@pytest.mark.parametrize("M", [1, 6, 16, 40])
def test_matvec_every_nibble_and_scale(nv, M):
    """One weight at a time: with a single non-zero activation the result is
    that weight (times it), whatever the nibble, the scale and the place in a row."""
    K = 256
    rng = np.random.Generator(np.random.PCG64(M))
    for fmt, codes in (("nvfp4", np.arange(127)), ("mxfp4", np.arange(0, 253))):
        block = 16 if fmt == "nvfp4" else 32
        N = len(codes)
        q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        q[:, :8] = np.arange(8) * 2 + ((np.arange(8) * 2 + 1) << 4)  # every nibble in every row
        s = np.repeat(codes.astype(np.uint8)[:, None], K // block, axis=1)
        w = values(q, s, fmt)
        at = np.concatenate([np.arange(16), rng.integers(16, K, 3)])
        for k in at[np.arange(0, 19, 1 if M == 1 else 6)]:
            x = np.zeros((M, K), np.float32)
            x[M - 1, k] = 1.0
            y = _run(nv, fmt, torch.from_numpy(x).bfloat16().to("cuda:0"), _dev(q), _dev(s), _gs(1.0), torch.float32)
            got = host(y).astype(np.float64)
            assert np.array_equal(got[M - 1], w[:, k]) and not got[:M - 1].any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [2, 7, 16, 50])
def test_matvec_tokens_do_not_touch_each_other(nv, fmt, M):
    """A token's infinite and NaN values stay its own."""
    K, N = 416, 70
    rng = np.random.Generator(np.random.PCG64(M))
    bits, _ = _x_bits(rng, M, K)
    q, s = weights(rng, N, K, fmt)
    x = dev_bf16(bits)
    clean = _run(nv, fmt, x, _dev(q), _dev(s), _gs(1.0), torch.float32)
    x[M - 1, 5], x[0, 400], x[0, 3] = float("inf"), float("nan"), -float("inf")
    got = _run(nv, fmt, x, _dev(q), _dev(s), _gs(1.0), torch.float32)
    assert torch.equal(got[1:M - 1], clean[1:M - 1])
    assert torch.isnan(got[0]).all() and not torch.isfinite(got[M - 1]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_matvec_writes_its_output_and_nothing_else(nv, dtype):
    rng = np.random.Generator(np.random.PCG64(2))
    for M, N in ((1, 17), (3, 33), (5, 31), (17, 47), (40, 65)):
        K = 224
        bits, x = _x_bits(rng, M, K)
        q, s = weights(rng, N, K, "mxfp4")
        room = torch.full((M * N + 2048,), 77.0, dtype=dtype, device="cuda:0")
        out = room[1024:1024 + M * N].view(M, N)
        assert nv.mx_matvec(dev_bf16(bits), _dev(q), _dev(s), out=out) is out
        w = values(q, s, "mxfp4")
        _check(out, x @ w.T, np.abs(x) @ np.abs(w).T, K, dtype)
        assert (room[:1024] == 77).all() and (room[1024 + M * N:] == 77).all()


def test_matvec_rows_are_those_of_the_linear_weights(nv):
    """The same weights as nvfp4_linear and mxfp4_linear take, x chosen so that
    quantizing it changes nothing: the two operators then agree to fp32 sums."""
    rng = np.random.Generator(np.random.PCG64(9))
    M, K, N = 6, 512, 256
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).bfloat16().to("cuda:0")
    x = torch.from_numpy(rng.choice([-6.0, -3.0, 0.5, 1.0, 6.0], (M, K)).astype(np.float32)).bfloat16().to("cuda:0")
    x[:, ::16] = 6.0
    for a, b in ((nv.matvec(x, *nv.quantize(w), out_dtype=torch.float32),
                  nv.linear(x, *nv.quantize(w), out_dtype=torch.float32, x_gs=_gs(1.0 / 448))),
                 (nv.mx_matvec(x, *nv.mx_quantize(w), out_dtype=torch.float32),
                  nv.mx_linear(x, *nv.mx_quantize(w), out_dtype=torch.float32))):
        mag = 6.0 * K * float(w.abs().max()) * 1.25
        assert float((a - b).abs().max()) <= 2 * (K + 2) * 2.0 ** -24 * mag + 1e-6 * float(b.abs().max())


def test_matvec_streams_and_graphs(nv):
    """On a stream of its own, and captured: every replay gives the eager result
    for what the inputs hold then."""
    rng = np.random.Generator(np.random.PCG64(4))
    cases = []
    for fmt, M, K, N in (("nvfp4", 1, 1024, 100), ("mxfp4", 5, 416, 61), ("nvfp4", 20, 640, 50)):
        q, s = weights(rng, N, K, fmt)
        cases.append((fmt, dev_bf16(_x_bits(rng, M, K)[0]), _dev(q), _dev(s), _gs(0.5)))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        on_stream = [_run(nv, *c, torch.float32) for c in cases]
    stream.synchronize()
    for c, y in zip(cases, on_stream):
        assert torch.equal(y, _run(nv, *c, torch.float32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [_run(nv, *c, torch.float32) for c in cases]
    for r in range(4):
        for c in cases:
            c[1].copy_(torch.randn(c[1].shape, device="cuda:0"))
        graph.replay()
        torch.cuda.synchronize()
        for c, y in zip(cases, outs):
            assert torch.equal(y, _run(nv, *c, torch.float32)), r


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M", [1, 4, 7, 16, 40])
def test_matvec_largest_and_smallest_values(nv, fmt, M):
    """Activations next to bf16's limit under scales that bring the results back
    into range, and subnormal ones: nothing overflows or is lost on the way."""
    rng = np.random.Generator(np.random.PCG64(M))
    K, N = 1184, 50
    q, _ = weights(rng, N, K, fmt)
    sign = (rng.integers(0, 2, (M, K)) << 15).astype(np.uint16)
    big = (0x7f00 | rng.integers(0, 128, (M, K), dtype=np.uint16) | sign) * (rng.integers(0, 64, (M, K)) == 5).astype(np.uint16)
    small = rng.integers(0, 0x300, (M, K), dtype=np.uint16) | sign
    # E4M3 scales of 2^-9 to 3 * 2^-9 and of 16 to 448, E8M0 of 2^-27 to 2^-10 and of 2^3 to 2^12
    for bits, codes in ((big, (1, 4) if fmt == "nvfp4" else (100, 118)), (small, (0x58, 0x7f) if fmt == "nvfp4" else (130, 140))):
        s = rng.integers(*codes, (N, K // (16 if fmt == "nvfp4" else 32)), dtype=np.uint8)
        x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double().numpy()
        w = values(q, s, fmt)
        ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        assert mag.max() < 2.0 ** 128
        got = _run(nv, fmt, dev_bf16(bits), _dev(q), _dev(s), _gs(1.0), torch.float32).double().cpu().numpy()
        assert (np.abs(got - ref) <= (K + 2) * (2.0 ** -24 * mag + 2.0 ** -149)).all()


@pytest.mark.parametrize("M", [1, 7, 16, 40])
@pytest.mark.parametrize("top,gs", [(106, 2.0 ** -100), (106, 2.0 ** -1), (-100, 2.0 ** 100)])
def test_matvec_tensor_scale_on_large_and_small_sums(nv, M, top, gs):
    """The tensor scale multiplies the finished sum: magnitudes up to 2^128 before it are right after it."""
    rng = np.random.Generator(np.random.PCG64(M))
    K, N = 1184, 50
    q, _ = weights(rng, N, K, "nvfp4")
    s = rng.integers(0x70, 0x7f, (N, K // 16), dtype=np.uint8)  # 128 to 448
    x = torch.from_numpy(rng.uniform(-1, 1, (M, K))).bfloat16().double().numpy() * 2.0 ** top
    w = values(q, s, "nvfp4")
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    assert mag.max() < 2.0 ** 128 and (top < 0 or mag.max() > 2.0 ** 124)
    got = nv.matvec(torch.from_numpy(x).bfloat16().to("cuda:0"), _dev(q), _dev(s), _gs(gs), out_dtype=torch.float32)
    _check(got, ref * gs, mag * gs, K, torch.float32)


def test_matvec_two_graphs_on_two_streams(nv):
    """Two captured calls of each kernel, replayed side by side: nothing is shared."""
    rng = np.random.Generator(np.random.PCG64(14))
    weight = weights(rng, 5000, 1056, "nvfp4")
    q, s = (_dev(a) for a in weight)
    gs = _gs(0.75)
    streams, graphs, outs, xs = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for i in range(2):
        xs.append([dev_bf16(_x_bits(rng, M, 1056)[0]) for M in (2, 7, 15, 30, 64)])
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            outs.append([nv.matvec(x, q, s, gs) for x in xs[i]])
    ref = [[nv.matvec(x, q, s, gs) for x in xs[i]] for i in range(2)]
    for _ in range(3):
        for i in range(2):
            for y in outs[i]:
                y.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i]))


def test_matvec_weights_beyond_4_gib(nv):
    """N * K / 2 = 4.5 GiB: the rows on both sides of 2^32 bytes."""
    K, N = 16384, 590000
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(3)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda:0", generator=gen)
    s = torch.randint(118, 126, (N, K // 32), dtype=torch.uint8, device="cuda:0", generator=gen)
    for M in (1, 3, 12):
        x = torch.randn(M, K, device="cuda:0", generator=gen).bfloat16()
        y = nv.mx_matvec(x, q, s, out_dtype=torch.float32)
        at = torch.tensor([0, 1, 524287, 524288, 524289, 550000, N - 2, N - 1], device="cuda:0")
        w = values(q[at].cpu().numpy(), s[at].cpu().numpy(), "mxfp4")
        xd = x.double().cpu().numpy()
        _check(y[:, at], xd @ w.T, np.abs(xd) @ np.abs(w).T, K, torch.float32)


def test_matvec_rejects_wrong_operands(nv):
    rng = np.random.Generator(np.random.PCG64(1))
    x = dev_bf16(_x_bits(rng, 2, 64)[0])
    q, s = (_dev(a) for a in weights(rng, 8, 64, "nvfp4"))
    with pytest.raises(ValueError, match="w_q"):
        nv.matvec(x, q[:, :16].contiguous(), s, _gs(1.0))
    with pytest.raises(ValueError, match="scales"):
        nv.mx_matvec(x, q, s)
    with pytest.raises(ValueError, match="w_gs"):
        nv.matvec(x, q, s, torch.ones(8, device="cuda:0"))
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        nv.matvec(x.float(), q, s, _gs(1.0))
    with pytest.raises(ValueError, match="contiguous"):
        nv.matvec(x.t().contiguous().t(), q, s, _gs(1.0))
    with pytest.raises(ValueError, match="output"):
        nv.matvec(x, q, s, _gs(1.0), out_dtype=torch.float16)
    with pytest.raises(nv.Nvfp4Error, match="K % 32"):
        nv.matvec(x[:, :48].contiguous(), q[:, :24].contiguous(), s[:, :3].contiguous(), _gs(1.0))
    assert nv.matvec(x[:0], q, s, _gs(1.0)).shape == (0, 8)
    assert host_bits(nv.matvec(x, q, s, _gs(0.0))).shape == (2, 8)
