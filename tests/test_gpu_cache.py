"""GPU parity of the quantized cache: bytes against the tensor quantizers (NVFP4,
MXFP4: themselves held to the oracle) and against a 64-bit search (MXFP8), reads
against the values of the bytes.  Reads of MX formats are exact in fp32; NVFP4
rounds once (the product with gs; e2m1 * sf is exact): half a step, 2^-24, and
2^-8 more for bf16 (2^-133 where results underflow)."""
import numpy as np
import pytest
import torch

from block_util import BLOCK, to_mxfp8, values, weights
from gpu_util import dev_bf16, host, host_bits

pytestmark = pytest.mark.gpu

FORMATS = ["nvfp4", "mxfp4", "mxfp8"]


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to("cuda:0")


def _gs(fmt, v=0.021):
    return torch.tensor([v], dtype=torch.float32, device="cuda:0") if fmt == "nvfp4" else None


def _rows(seed, T, shape):
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)
    spread = torch.exp(2 * torch.randn(shape, generator=gen, device="cuda:0"))
    return (torch.randn((T, *shape), generator=gen, device="cuda:0") * spread).bfloat16()


def _bytes(nv, x, fmt, gs):
    """The quantized form of rows, by the tensor quantizers or the definition."""
    flat = x.reshape(x.shape[0], -1).contiguous()
    if fmt == "nvfp4":
        q, s, _ = nv.quantize(flat, gs=gs)
    elif fmt == "mxfp4":
        q, s = nv.mx_quantize(flat)
    else:
        q, s = (torch.from_numpy(a).to(x.device) for a in to_mxfp8(flat.double().cpu().numpy()))
    return q.view(*x.shape[:-1], -1), s.view(*x.shape[:-1], -1)


def _same_values(got, q, s, fmt, gs, dtype):
    ref = values(host(q), host(s), fmt, 1.0 if gs is None else float(gs))
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    tol = np.abs(ref) * (2.0 ** -24 if fmt == "nvfp4" else 0.0) + (2.0 ** -149 if fmt == "nvfp4" else 0.0)
    if dtype == torch.bfloat16:
        tol = tol + np.abs(ref) * 2.0 ** -8 + 2.0 ** -134
    assert (np.abs(got - ref) <= tol).all()


SHAPES = [(1, (8, 128)), (5, (576,)), (130, (3, 96)), (33, (1, 32)), (257, (2, 64)), (1025, (64,)), (7, (16, 256)),
          (4099, (4, 160))]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,shape", SHAPES)
def test_cache_write_and_read(nv, fmt, T, shape):
    rng = np.random.Generator(np.random.PCG64(T))
    n = 2 * T + 3
    gs = _gs(fmt)
    x = _rows(T, T, shape)
    cache = nv.cache_empty(n, shape, fmt, "cuda:0", gs)
    for t in cache[:2]:
        t.fill_(0x5a)
    slots = rng.permutation(n)[:T].astype(np.int32)
    off = rng.random(T) < 0.2
    if T > 1:
        slots[off] = rng.choice([-1, n, -2 ** 31, 2 ** 31 - 1], off.sum())
    else:
        off[:] = False
    assert nv.cache_write(x, _i32(slots), cache, format=fmt) is None
    q, s = _bytes(nv, x, fmt, gs)
    want_q, want_s = torch.full_like(cache[0], 0x5a), torch.full_like(cache[1], 0x5a)
    on = torch.from_numpy(~off).to("cuda:0")
    want_q[_i32(slots).long()[on]] = q[on]
    want_s[_i32(slots).long()[on]] = s[on]
    assert torch.equal(cache[0], want_q) and torch.equal(cache[1], want_s)
    for dtype in (torch.bfloat16, torch.float32):
        back = nv.cache_read(cache, _i32(slots), format=fmt, out_dtype=dtype)
        assert back.dtype == dtype and tuple(back.shape) == (T, *shape)
        _same_values(back[on], q[on], s[on], fmt, gs, dtype)
        assert not back[~on].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_cache_keys_and_values_of_a_fused_projection(nv, fmt):
    """Two parts with rows of different lengths, columns of one matrix."""
    T, hk, hv, n = 77, (4, 96), (4, 64), 100
    fused = _rows(3, T, (2 * 384 + 384 + 256,))
    k, v = fused[:, 768:1152].unflatten(1, hk), fused[:, 1152:].unflatten(1, hv)
    gs = _gs(fmt)
    caches = [nv.cache_empty(n, h, fmt, "cuda:0", gs) for h in (hk, hv)]
    slots = _i32(np.random.Generator(np.random.PCG64(1)).permutation(n)[:T])
    nv.cache_write((k, v), slots, caches, format=fmt)
    got = nv.cache_read(caches, slots, format=fmt)
    assert isinstance(got, tuple) and len(got) == 2
    for t, c, y in zip((k, v), caches, got):
        q, s = _bytes(nv, t, fmt, gs)
        assert torch.equal(c[0][slots.long()], q) and torch.equal(c[1][slots.long()], s)
        _same_values(y, q, s, fmt, gs, torch.bfloat16)


def test_mxfp8_every_bf16_value(nv):
    """Every finite bf16 magnitude as a block's maximum and, under several
    maxima, as an element, against the 64-bit search."""
    bits = np.arange(0x7f80, dtype=np.uint16)
    rng = np.random.Generator(np.random.PCG64(5))
    tops = np.zeros((len(bits), 32), np.uint16)
    tops[:, 0] = bits
    tops[:, 1:] = np.minimum(rng.integers(0, 0x7f80, (len(bits), 31)), bits[:, None]) | (
        rng.integers(0, 2, (len(bits), 31)) << 15).astype(np.uint16)
    elements = np.concatenate([np.resize(bits, (1053, 31)), np.resize(bits | 0x8000, (1053, 31))]).astype(np.uint16)
    blocks = [tops]
    for top in (0x0001, 0x0460, 0x3f80, 0x3fe0, 0x3fe1, 0x3fff, 0x7f7f):
        e = elements.copy()
        e[(e & 0x7fff) > top] &= 0x8000
        blocks.append(np.concatenate([np.full((len(e), 1), top, np.uint16), e], axis=1))
    x = np.concatenate(blocks)
    d = dev_bf16(x)
    cache = nv.cache_empty(len(x), (32,), device="cuda:0")
    at = torch.arange(len(x), dtype=torch.int32, device="cuda:0")
    nv.cache_write(d, at, cache)
    q, s = to_mxfp8(d.double().cpu().numpy())
    assert np.array_equal(host(cache[1]), s)
    assert np.array_equal(host(cache[0]), q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_mxfp8_largest_values_come_back_finite(nv, dtype):
    """The bf16 values whose blocks have the largest code a write makes, 247: the
    elements that are rounded up to 2^128 are read as bf16's largest value, all
    within half a step, 2^-4; then every element byte under every code from there on."""
    top = np.arange(0x7f00, 0x7f80, dtype=np.uint16)
    x = np.zeros((2 * len(top), 32), np.uint16)
    x[:, 0] = np.concatenate([top, top | 0x8000])
    x[:, 1:] = np.resize(np.concatenate([top[::-1], np.arange(0, 0x7f80, 0x155, dtype=np.uint16)]), (len(x), 31))
    x[:, 1:] = np.minimum(x[:, 1:], x[:, :1] & 0x7fff) | (np.arange(31) % 2 << 15).astype(np.uint16)
    d = dev_bf16(x)
    cache = nv.cache_empty(len(x), (32,), device="cuda:0")
    at = torch.arange(len(x), dtype=torch.int32, device="cuda:0")
    nv.cache_write(d, at, cache)
    assert int(cache[1].max()) == 247
    largest = 255 / 128 * 2.0 ** 127
    got = nv.cache_read(cache, at, out_dtype=dtype).double().cpu().numpy()
    assert np.array_equal(got, np.clip(values(host(cache[0]), host(cache[1]), "mxfp8"), -largest, largest))
    xd = d.double().cpu().numpy()
    assert (np.abs(got - xd) <= np.maximum(np.abs(xd) * 2.0 ** -4, 2.0 ** 120 * 2.0 ** -10)).all()
    codes = np.arange(247, 255)
    q = np.tile(np.arange(256, dtype=np.uint8), (len(codes), 1))
    s = np.repeat(codes.astype(np.uint8)[:, None], 8, axis=1)
    cache = torch.from_numpy(q).to("cuda:0"), torch.from_numpy(s).to("cuda:0")
    got = nv.cache_read(cache, at[:len(codes)], out_dtype=dtype).double().cpu().numpy()
    assert np.array_equal(got, np.clip(values(q, s, "mxfp8"), -largest, largest), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_cache_read_every_byte(nv, dtype):
    """Every element byte under every scale byte of each format (values inside
    fp32; bf16 rounds to nearest even)."""
    for fmt, codes in (("mxfp8", np.arange(0, 247)), ("mxfp4", np.arange(0, 253)), ("nvfp4", np.arange(127))):
        n = len(codes)
        q = np.tile(np.arange(256, dtype=np.uint8), (n, 1))
        if fmt == "mxfp8":
            q[:, 127], q[:, 255] = 0, 0  # NaN patterns, which a write never leaves
        blocks = (256 if fmt == "mxfp8" else 512) // BLOCK[fmt]
        s = np.repeat(codes.astype(np.uint8)[:, None], blocks, axis=1)
        gs = _gs(fmt, 0.37)
        cache = tuple(t for t in (torch.from_numpy(q).to("cuda:0"), torch.from_numpy(s).to("cuda:0"), gs) if t is not None)
        at = torch.arange(n, dtype=torch.int32, device="cuda:0")
        got = nv.cache_read(cache, at, format=fmt, out_dtype=dtype)
        f32 = values(q, s, fmt)
        if fmt == "nvfp4":
            f32 = (f32.astype(np.float32) * np.float32(0.37)).astype(np.float32)
        want = torch.from_numpy(f32.astype(np.float32))
        assert np.array_equal(f32.astype(np.float32).astype(np.float64), f32)
        assert torch.equal(got.cpu(), want.to(dtype))


def _table(rng, lens, page, pool, wide):
    need = [-(-n // page) for n in lens]
    free = list(rng.permutation(pool))
    table = np.full((len(lens), wide), -1, np.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = free.pop()
    return table


LENS = [([1], 1), ([0, 1, 0, 17, 64, 0], 16), ([5, 300, 0, 0, 129], 64), ([3, 2, 1], 7), ([0, 0], 4),
        ([700, 1, 1, 33, 0, 255, 256, 257], 256), ([1] * 40 + [0] * 30 + [9], 8)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,page", LENS)
def test_cache_read_pages(nv, fmt, lens, page):
    rng = np.random.Generator(np.random.PCG64(len(lens)))
    shape = (2, 96)
    pool = sum(-(-n // page) for n in lens) + 3
    wide = max(1, max(-(-n // page) for n in lens)) + 1
    table = _table(rng, lens, page, pool, wide)
    q, s = weights(rng, pool * page * 2, 96, fmt if fmt != "mxfp8" else "mxfp4")
    if fmt == "mxfp8":
        q = rng.integers(0, 127, (pool * page * 2, 96), dtype=np.uint8)
    q, s = q.reshape(pool * page, 2, -1), s.reshape(pool * page, 2, -1)
    gs = _gs(fmt)
    cache = tuple(t for t in (torch.from_numpy(q).to("cuda:0"), torch.from_numpy(s).to("cuda:0"), gs) if t is not None)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    slots = np.array([table[b, i // page] * page + i % page for b, n in enumerate(lens) for i in range(n)], np.int64)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((total + 5, *shape), 9.0, dtype=dtype, device="cuda:0")
        got = nv.cache_read_pages(cache, _i32(table), _i32(cu), page, total + 5, format=fmt, out_dtype=dtype, out=out)
        assert got is out and (out[total:] == 9).all()
        if total:
            at = torch.from_numpy(slots).to("cuda:0")
            _same_values(out[:total], cache[0][at], cache[1][at], fmt, gs, dtype)
            assert torch.equal(out[:total], nv.cache_read(cache, at.int(), format=fmt, out_dtype=dtype))


def test_cache_read_pages_outside_the_table(nv):
    """Pages outside the cache, sequences longer than the table's rows, lengths
    that start behind row 0: zeros, or left as they were; nothing is read out of range."""
    cache = nv.cache_empty(40, (32,), device="cuda:0")
    x = _rows(1, 40, (32,)).abs() + 1
    nv.cache_write(x, torch.arange(40, dtype=torch.int32, device="cuda:0"), cache)
    full = nv.cache_read(cache, torch.arange(40, dtype=torch.int32, device="cuda:0"))
    table = np.array([[3, -1], [10, 9], [2 ** 31 - 1, 0], [-2 ** 31, 1]], np.int32)  # page size 4: pages 0 .. 9
    cu = np.array([2, 10, 22, 30, 38], np.int32)  # the second sequence has 12 rows, its table row holds 8
    out = torch.full((41, 32), 9.0, dtype=torch.bfloat16, device="cuda:0")
    nv.cache_read_pages(cache, _i32(table), _i32(cu), 4, 41, out=out)
    want = torch.zeros_like(out)
    want[:2], want[38:] = 9.0, 9.0
    want[2:6], want[14:18], want[26:30], want[34:38] = full[12:16], full[36:40], full[0:4], full[4:8]
    assert torch.equal(out, want)


def test_cache_read_pages_of_many_sequences(nv):
    """More than 2^30 sequences, nearly all of them empty: the search for a row's
    sequence goes through indices whose sums pass 2^31."""
    B, at = 2 ** 30 + 5, 2 ** 30 + 2
    cache = nv.cache_empty(16, (32,), device="cuda:0")
    nv.cache_write(_rows(1, 16, (32,)).abs() + 1, torch.arange(16, dtype=torch.int32, device="cuda:0"), cache)
    full = nv.cache_read(cache, torch.arange(16, dtype=torch.int32, device="cuda:0"))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda:0")
    cu[at + 1:], cu[B] = 1, 2
    pages = torch.zeros(B, 1, dtype=torch.int32, device="cuda:0")
    pages[at], pages[B - 1] = 3, 1
    got = nv.cache_read_pages(cache, pages, cu, 4, 2)
    assert torch.equal(got, full[[12, 4]])


def test_cache_beyond_4_gib(nv):
    """4.6 GiB of elements: slots on both sides of 2^32 bytes."""
    shape, n = (8, 128), 4_800_000
    cache = nv.cache_empty(n, shape, device="cuda:0")
    at = [0, 1, 4194303, 4194304, 4194305, 4500000, n - 1]
    x = _rows(2, len(at), shape)
    nv.cache_write(x, _i32(at), cache)
    q, s = _bytes(nv, x, "mxfp8", None)
    assert torch.equal(cache[0][torch.tensor(at, device="cuda:0")], q)
    assert torch.equal(cache[1][torch.tensor(at, device="cuda:0")], s)
    assert int((cache[1] != 0).sum()) == int((s != 0).sum())
    _same_values(nv.cache_read(cache, _i32(at)), q, s, "mxfp8", None, torch.bfloat16)
    pages = _i32([[n // 16 - 1, 4194304 // 16]])
    got = nv.cache_read_pages(cache, pages, _i32([0, 17]), 16, 17)
    assert torch.equal(got[15], nv.cache_read(cache, _i32([n - 1]))[0])
    assert torch.equal(got[16], nv.cache_read(cache, _i32([4194304]))[0])


def test_cache_skipped_rows_may_hold_anything(nv):
    for fmt in FORMATS:
        x = _rows(4, 6, (2, 64))
        x[2], x[5] = float("nan"), float("inf")
        cache = nv.cache_empty(9, (2, 64), fmt, "cuda:0", _gs(fmt))
        nv.cache_write(x, _i32([4, 0, -1, 8, 3, 9]), cache, format=fmt)
        q, s = _bytes(nv, x[[0, 1, 3, 4]].contiguous(), fmt, _gs(fmt))
        assert torch.equal(cache[0][[4, 0, 8, 3]], q) and torch.equal(cache[1][[4, 0, 8, 3]], s)
        assert not cache[0][[1, 2, 5, 6, 7]].any() and not cache[1][[1, 2, 5, 6, 7]].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_cache_infinite_and_nan_values_stay_in_their_block(nv, fmt):
    T, shape, block = 9, (3, 96), BLOCK[fmt]
    gs = _gs(fmt)
    x, at = _rows(8, T, shape), torch.arange(T, dtype=torch.int32, device="cuda:0")
    caches = [nv.cache_empty(T, shape, fmt, "cuda:0", gs) for _ in range(2)]
    nv.cache_write(x, at, caches[0], format=fmt)
    hit = torch.zeros(T, 3, 96 // block, dtype=torch.bool, device="cuda:0")
    for t, h, k, v in ((0, 0, 0, float("inf")), (2, 1, 50, float("nan")), (2, 2, 95, -float("inf")), (8, 2, 31, float("nan")),
                       (5, 0, 32, float("inf")), (5, 0, 33, float("nan"))):
        x[t, h, k] = v
        hit[t, h, k // block] = True
    nv.cache_write(x, at, caches[1], format=fmt)
    for a, b in zip(caches[0][:2], caches[1][:2]):
        a, b = (c.unflatten(-1, (96 // block, -1))[~hit] for c in (a, b))
        assert torch.equal(a, b)


def test_cache_streams_and_graphs(nv):
    """Written and read on a stream of its own, and captured: every replay
    writes and reads what the inputs hold then, padding included."""
    T, shape, n = 21, (3, 64), 64
    x, slots = _rows(6, T, shape), _i32(np.arange(T))
    pages, cu = _i32([[0, 1], [2, 3]]), _i32([0, 20, 30])
    caches = {f: nv.cache_empty(n, shape, f, "cuda:0", _gs(f)) for f in FORMATS}
    other = {f: nv.cache_empty(n, shape, f, "cuda:0", _gs(f)) for f in FORMATS}
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for f in FORMATS:
            nv.cache_write(x, slots, other[f], format=f)
        rows = {f: nv.cache_read(other[f], slots, format=f) for f in FORMATS}
    stream.synchronize()
    for f in FORMATS:
        nv.cache_write(x, slots, caches[f], format=f)
        assert torch.equal(caches[f][0], other[f][0]) and torch.equal(rows[f], nv.cache_read(caches[f], slots, format=f))
    outs = {f: torch.zeros((32, *shape), dtype=torch.bfloat16, device="cuda:0") for f in FORMATS}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in FORMATS:
            nv.cache_write(x, slots, caches[f], format=f)
            nv.cache_read_pages(caches[f], pages, cu, 16, 32, format=f, out=outs[f])
    rng = np.random.Generator(np.random.PCG64(3))
    for r in range(4):
        x.copy_(_rows(10 + r, T, shape))
        at = rng.permutation(n)[:T].astype(np.int32)
        at[T - r:] = -1
        slots.copy_(_i32(at))
        pages.copy_(_i32(rng.permutation(4).reshape(2, 2)))
        cu.copy_(_i32([0, 16 + r, 25 + r]))
        graph.replay()
        torch.cuda.synchronize()
        for f in FORMATS:
            nv.cache_write(x, slots, other[f], format=f)
            assert torch.equal(caches[f][0], other[f][0]) and torch.equal(caches[f][1], other[f][1]), r
            want = nv.cache_read_pages(other[f], pages, cu, 16, 32, format=f)[:25 + r]
            assert torch.equal(outs[f][:25 + r], want), r


def test_projection_cache_and_back(nv):
    """A decode step's use of the operators together: the fused projection of
    eight requests with 4-bit weights, their keys and values into the cache, all
    rows of the requests back by page table; eager and captured."""
    B, K, hq, h, dim, page = 8, 1024, 8, 2, 128, 16
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(11)
    w = (torch.randn((hq + 2 * h) * dim, K, generator=gen, device="cuda:0") * 0.05).bfloat16()
    wq = nv.quantize(w)
    lens = np.array([0, 1, 15, 16, 17, 40, 31, 32])
    table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)[:, ::-1].copy()
    caches = [nv.cache_empty(B * 4 * page, (h, dim), device="cuda:0") for _ in range(2)]
    total = int(lens.sum())
    past = [_rows(20 + i, total, (h, dim)) for i in range(2)]
    before = np.array([table[b, i // page] * page + i % page for b in range(B) for i in range(lens[b])])
    nv.cache_write(past, _i32(before), caches)
    slots = _i32([table[b, lens[b] // page] * page + lens[b] % page for b in range(B)])
    cu = _i32(np.concatenate([[0], np.cumsum(lens + 1)]))
    pages = _i32(table)
    x = torch.randn(B, K, generator=gen, device="cuda:0").bfloat16()

    def step(x):
        y = nv.matvec(x, *wq)
        k, v = y[:, hq * dim:(hq + h) * dim].unflatten(1, (h, dim)), y[:, (hq + h) * dim:].unflatten(1, (h, dim))
        nv.cache_write((k, v), slots, caches)
        return y, nv.cache_read_pages(caches, pages, cu, page, total + B)

    def check(x, y, back):
        ref = x.double() @ nv.dequantize(*wq, out_dtype=torch.float32).double().t().contiguous()
        mag = x.double().abs() @ nv.dequantize(*wq, out_dtype=torch.float32).double().abs().t().contiguous()
        tol = (K + 2) * 2.0 ** -23 * mag + ref.abs() * 2.0 ** -8  # one more rounding: the dequantized weights'
        assert ((y.double() - ref).abs() <= tol).all()
        for i, (p, b) in enumerate(zip(past, back)):
            at = hq * dim + i * h * dim
            new = y[:, at:at + h * dim].unflatten(1, (h, dim))
            ends = np.cumsum(lens)
            rows = torch.cat([torch.cat([p[ends[s] - lens[s]:ends[s]], new[s:s + 1]]) for s in range(B)])
            q, sc = _bytes(nv, rows, "mxfp8", None)
            _same_values(b, q, sc, "mxfp8", None, torch.bfloat16)

    check(x, *step(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, back = step(x)
    for _ in range(3):
        x.copy_(torch.randn(B, K, generator=gen, device="cuda:0"))
        graph.replay()
        torch.cuda.synchronize()
        check(x, y, back)


def test_cache_rejects_wrong_operands(nv):
    cache = nv.cache_empty(8, (2, 64), device="cuda:0")
    x, slots = _rows(1, 4, (2, 64)), _i32([0, 1, 2, 3])
    with pytest.raises(ValueError, match="rows must be"):
        nv.cache_write(x[:3], slots, cache)
    with pytest.raises(ValueError, match="rows must be"):
        nv.cache_write(x.float(), slots, cache)
    with pytest.raises(ValueError, match="contiguous"):
        nv.cache_write(x.transpose(1, 2).contiguous().transpose(1, 2), slots, cache)
    with pytest.raises(ValueError, match="slots"):
        nv.cache_write(x, slots.long(), cache)
    with pytest.raises(ValueError, match=r"\(q, s"):
        nv.cache_write(x, slots, cache, format="nvfp4")
    with pytest.raises(ValueError, match="must be"):
        nv.cache_write(x, slots, cache, format="mxfp4")
    with pytest.raises(ValueError, match="tensors for"):
        nv.cache_write([x], slots, [cache, cache])
    with pytest.raises(nv.Nvfp4Error, match="overlap"):
        nv.cache_write((x, x), slots, (cache, cache))
    with pytest.raises(nv.Nvfp4Error, match="multiple of 8"):
        nv.cache_write(torch.zeros(4, 133, dtype=torch.bfloat16, device="cuda:0")[:, :128].unflatten(1, (2, 64)), slots,
                       cache)
    with pytest.raises(ValueError, match="slots"):
        nv.cache_write((x, x), slots, (cache, nv.cache_empty(9, (2, 64), device="cuda:0")))
    with pytest.raises(ValueError, match="out must be"):
        nv.cache_read(cache, slots, out=torch.empty(4, 2, 32, dtype=torch.bfloat16, device="cuda:0"))
    with pytest.raises(ValueError, match="out"):
        nv.cache_read(cache, slots, out=torch.empty(4, 2, 64, device="cuda:0"))
    with pytest.raises(ValueError, match="cu_lens"):
        nv.cache_read_pages(cache, _i32([[0]]), _i32([0]), 4, 1)
    assert nv.cache_read(cache, slots[:0]).shape == (0, 2, 64)
    assert host_bits(nv.cache_read(nv.cache_empty(0, (2, 64), device="cuda:0"), slots)).any() == 0
