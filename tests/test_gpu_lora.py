"""Low-rank adapters of many requests on the GPU against the definition in 64
bits, and in a run with the projections, the router and the expert FFN."""
import pytest
import torch

import synth
from gpu_util import dev_f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _ids(kind, T, L, g):
    if kind == "one":
        i = torch.full((T,), L - 1)
    elif kind == "none":
        i = torch.full((T,), -1)
    elif kind == "requests":  # runs of tokens, some of them without an adapter
        i = torch.sort(torch.randint(-1, L, (T,), generator=g)).values.roll(T // 3)
    elif kind == "distinct":
        i = torch.randperm(max(T, L), generator=g)[:T] % L
    else:                     # tokens of all adapters mixed, ids outside the range on either side
        i = torch.randint(-3, L + 3, (T,), generator=g)
    return i.to(torch.int32)


def _problem(T, K, N, r, L, dtype, kind, seed):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(T, N, generator=g).to(dtype)
    x = torch.randn(T, K, generator=g).to(BF)
    a = (torch.randn(L, r, K, generator=g) / K ** 0.5).to(BF)
    b = (torch.randn(L, N, r, generator=g) * 0.5).to(BF)
    s = torch.rand(L, generator=g) * 2 - 0.5
    return [v.to(DEV) for v in (y, x, a, b, _ids(kind, T, L, g), s)]


def _definition(y, x, a, b, ids, s):
    """(result, largest magnitude of the delta's terms, mean square of all terms)"""
    want = y.double()
    size, square = torch.zeros_like(want), want.square()
    for l in range(a.shape[0]):
        t = torch.nonzero(ids == l).flatten()
        if t.numel():
            f = 1.0 if s is None else float(s[l])
            xd, ad, bd = x[t].double(), a[l].double().t().contiguous(), b[l].double().t().contiguous()
            want[t] += f * ((xd @ ad) @ bd)
            size[t] = abs(f) * ((xd.abs() @ ad.abs()) @ bd.abs())
            square[t] += f * f * ((xd.square() @ ad.square()) @ bd.square())
    return want, size, square


def _check(out, y, x, a, b, ids, s):
    """Per element: the output's rounding (half a step of it, and of the sum it
    rounds), K + 64 roundings of the first sum and 3 r + 16 of the second
    (three terms of u), no partial sum over the sum of its terms' magnitudes;
    u as two (bf16 output) or three bf16 terms leaves 2^-16 or 2^-24 of it.
    For fp32 outputs also over all elements: a walk of K / 8 + 3 r / 8 + 24
    roundings as uniform errors of partial sums whose mean square is at most
    that of all terms, allowed twice."""
    K, r = x.shape[1], a.shape[1]
    want, size, square = _definition(y, x, a, b, ids, s)
    half = torch.finfo(y.dtype).eps / 2
    rest = 2.0 ** -16 if y.dtype == BF else 2.0 ** -24
    tol = half * 1.001 * want.abs() + size * ((K + 64 + 3 * r + 16) * 2.0 ** -24 + rest) * 1.01
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), torch.nonzero(err > tol)[:4])
    bare = (ids < 0) | (ids >= a.shape[0])
    assert torch.equal(out[bare], y[bare])
    if y.dtype == torch.float32:
        rel = float(err.norm() / square.sum().sqrt())
        assert rel <= 2 * ((K / 8 + 3 * r / 8 + 24) / 3) ** 0.5 * 2.0 ** -24, rel


SHAPES = [(1, 32, 8, 8, 1), (1, 7168, 2048, 16, 4), (2, 64, 24, 16, 2), (15, 96, 72, 24, 3), (16, 160, 264, 32, 5),
          (17, 1280, 256, 40, 2), (65, 512, 1000, 64, 40), (100, 768, 512, 128, 7), (300, 256, 136, 96, 512),
          (1000, 128, 96, 8, 9), (1024, 64, 64, 16, 64), (1025, 64, 320, 48, 6), (1500, 512, 264, 16, 3),
          (4097, 96, 40, 56, 33), (5003, 256, 128, 64, 5), (256, 2048, 96, 32, 3), (257, 1024, 48, 128, 2),
          (500, 4096, 40, 16, 20), (513, 512, 600, 104, 1)]


@pytest.mark.parametrize("T,K,N,r,L", SHAPES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_lora_shapes(nv, T, K, N, r, L, dtype):
    for i, kind in enumerate(("one", "requests", "mixed")):
        p = _problem(T, K, N, r, L, dtype, kind, T + 7 * i)
        keep = p[0].clone()
        _check(nv.lora_add(*p[:5], scales=p[5]), *p)
        assert torch.equal(p[0], keep)  # y itself is left alone
        p[5] = None
        out = torch.full_like(p[0], 3.0)
        assert nv.lora_add(*p[:5], out=out) is out
        _check(out, *p)


@pytest.mark.parametrize("T", [1, 40, 256, 257, 1024, 2100])
@pytest.mark.parametrize("kind", ["one", "none", "requests", "distinct", "mixed"])
def test_lora_ids(nv, T, kind):
    p = _problem(T, 128, 200, 16, 37, BF, kind, T)
    _check(nv.lora_add(*p[:5], scales=p[5]), *p)


@pytest.mark.parametrize("T,K,L", [(16384, 64, 512), (16384, 64, 3), (16385, 64, 5), (17000, 96, 512)])
@pytest.mark.parametrize("kind", ["one", "requests", "mixed"])
def test_lora_many_tokens(nv, T, K, L, kind):
    """The groupings of one and of many workgroups at their border."""
    p = _problem(T, K, 16, 8, L, BF, kind, T + L)
    _check(nv.lora_add(*p[:5], scales=p[5]), *p)
    y = p[0].clone()
    nv.lora_add(y, *p[1:5], scales=p[5], out=y)
    assert torch.equal(y, nv.lora_add(*p[:5], scales=p[5]))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T", [9, 3000])
def test_lora_in_place(nv, T, dtype):
    """In place gives the bits of the copying call, and rows without an adapter
    are not touched, whatever they hold."""
    p = _problem(T, 192, 104, 16, 4, dtype, "mixed", 3)
    bare = torch.nonzero((p[4] < 0) | (p[4] >= 4)).flatten()
    p[0][bare[0]] = float("nan")
    p[1][bare[0]] = float("inf")
    out = nv.lora_add(*p[:5], scales=p[5])
    y = p[0].clone()
    assert nv.lora_add(y, *p[1:5], scales=p[5], out=y) is y
    bits = torch.int16 if dtype == BF else torch.int32
    assert torch.equal(y.view(bits), out.view(bits))
    assert torch.equal(y[bare].view(bits), p[0][bare].view(bits))


@pytest.mark.parametrize("T", [50, 2000])
def test_lora_rows_are_independent(nv, T):
    """A token with NaN activations, and an adapter with infinite weights, spoil
    their own rows only."""
    p = _problem(T, 128, 96, 16, 6, BF, "requests", 5)
    p[4][:6] = torch.arange(6, dtype=torch.int32)
    good = nv.lora_add(*p[:5], scales=p[5])
    p[1][3] = float("nan")
    p[2][5] = float("inf")
    out = nv.lora_add(*p[:5], scales=p[5])
    keep = p[4] != 5
    keep[3] = False
    assert torch.equal(out[keep], good[keep])
    assert bool(torch.isnan(out[3]).all())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T,L", [(5, 2), (100, 2), (300, 2), (300, 40)])
def test_lora_infinite_activation(nv, T, L, dtype):
    """An infinite x with positive adapters gives an infinite row, as the sum
    does, and leaves the other rows bit for bit."""
    y, x, a, b, ids, _ = _problem(T, 256, 136, 8, L, dtype, "mixed", 11)
    a, b = a.abs() + 2.0 ** -6, b.abs() + 2.0 ** -6
    ids[T // 2] = L - 1
    want = nv.lora_add(y, x, a, b, ids)
    x[T // 2, 77] = float("inf")
    out = nv.lora_add(y, x, a, b, ids)
    assert torch.isposinf(out[T // 2]).all()
    rest = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(out[rest], want[rest])


def test_lora_repeats_bit_for_bit(nv):
    p = _problem(3000, 512, 512, 32, 9, torch.float32, "mixed", 8)
    first = nv.lora_add(*p[:5], scales=p[5])
    for _ in range(3):
        assert torch.equal(nv.lora_add(*p[:5], scales=p[5]), first)


def test_lora_large_offsets(nv):
    """Rows and adapters that lie behind 4 GiB."""
    T, N, K, r, L = 70000, 16384, 64, 8, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    y = torch.randn(T, N, generator=g, device=DEV)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    a = torch.randn(L, r, K, generator=g, device=DEV).to(BF)
    b = torch.randn(L, N, r, generator=g, device=DEV).to(BF)
    ids = (torch.arange(T, device=DEV) % 5 - 1).to(torch.int32)
    out = nv.lora_add(y, x, a, b, ids)
    rows = torch.tensor([0, 1, 2, 3, 33333, 65535, 65536, 65540, 69996, 69997, 69998, 69999], device=DEV)
    _check(out[rows], y[rows], x[rows], a, b, ids[rows], None)


@pytest.mark.parametrize("T", [24, 1800])
def test_lora_graph_and_streams(nv, T):
    """Captured once, replayed on new activations and new requests, with eager
    calls on the same and on another stream in between."""
    K, N, r, L = 256, 256, 16, 8
    p = _problem(T, K, N, r, L, BF, "mixed", 1)
    nv.lora_add(*p[:5], scales=p[5])
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = nv.lora_add(*p[:5], scales=p[5])
    ws = nv.lora_add_workspace(T, N, K, r, L, DEV)
    with torch.cuda.graph(g2):
        out2 = nv.lora_add(*p[:5], scales=p[5], ws=ws)
    side = torch.cuda.Stream()
    for i in range(4):
        q = _problem(T, K, N, r, L, BF, ("requests", "one", "none", "mixed")[i], 50 + i)
        for dst, src in zip(p, q):
            dst.copy_(src)
        g.replay()
        eager = nv.lora_add(*p[:5], scales=p[5])
        g2.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = nv.lora_add(*p[:5], scales=p[5])
        torch.cuda.synchronize()
        _check(eager, *p)
        for v in (out, out2, other):
            assert torch.equal(v, eager), i


def test_lora_refuses_bad_tensors(nv):
    y, x, a, b, ids, s = _problem(8, 64, 64, 16, 3, BF, "one", 0)
    for args, kw in (((y, x, a, b, ids.long()), {}), ((y, x.float(), a, b, ids), {}), ((y.half(), x, a, b, ids), {}),
                     ((y, x[:7], a, b, ids), {}), ((y, x, a, b[:2], ids), {}), ((y, x, a[:, :8].contiguous(), b, ids), {}),
                     ((y, x, a, b, ids[:7]), {}), ((y, x, a, b, ids), dict(scales=s[:2])),
                     ((y, x, a, b, ids), dict(out=torch.empty(8, 64, device=DEV))),
                     ((y, x, a, b, ids.cpu()), {}), ((y.t(), x, a, b, ids), {}),
                     ((y, x, a.transpose(1, 2), b, ids), {})):
        with pytest.raises(ValueError):
            nv.lora_add(*args, **kw)
    with pytest.raises(nv.Nvfp4Error):  # a rank that is no multiple of 8
        nv.lora_add(y, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ids)
    big = torch.empty(16, 64, dtype=BF, device=DEV)
    with pytest.raises(nv.Nvfp4Error, match="overlap"):
        nv.lora_add(big[:8], x, a, b, ids, out=big[4:12])
    assert nv.lora_add(y[:0], x[:0], a, b, ids[:0]).shape == (0, 64)


def test_lora_beside_the_projection_the_router_and_the_experts(nv):
    """A run as a serving step makes it: an NVFP4 projection with the requests'
    adapters, the gate, the routing, the expert FFN; eager and captured, the
    captured one replayed on new tokens and requests."""
    cfg = synth.TINY
    T, H, E, r, L = cfg.T, cfg.H, cfg.E, 16, 4
    g = torch.Generator().manual_seed(0)
    wq = nv.quantize((torch.randn(H, H, generator=g) * 0.06).to(BF).to(DEV))
    ew = [synth.expert_weights(cfg, e, device=DEV) for e in range(E)]
    w1 = nv.quantize_experts(torch.stack([v for v, _ in ew]))
    w2 = nv.quantize_experts(torch.stack([v for _, v in ew]))
    gate, a2 = (torch.randn(E, H, generator=g) * 0.1).to(DEV), dev_f32(cfg.a2_gs)
    _, x, a, b, ids, s = _problem(T, H, H, r, L, BF, "requests", 2)
    n = torch.tensor([T - 5], dtype=torch.int32, device=DEV)

    def step():
        h = nv.linear(x, *wq)
        base = h.clone()
        nv.lora_add(h, x, a, b, ids, scales=s, out=h)
        z = nv.router_logits(h, gate)
        e, w = nv.route(z, cfg.topk, scoring="sigmoid", n_group=2, topk_group=1, group_top=2, n_tokens=n)
        return base, h, z, e, w, nv.moe_expert_ffn(h, e, w, *w1, *w2, a2)

    base, h, z, e, w, y = step()
    torch.cuda.synchronize()
    _check(h, base, x, a, b, ids, s)
    zd = h.double() @ gate.double().t().contiguous()
    assert float((z - zd).norm() / zd.norm()) <= (H + 64) * 2.0 ** -24
    assert bool((e[:T - 5] >= 0).all()) and bool((e[T - 5:] == -1).all()) and bool((y[T - 5:] == 0).all())
    assert bool((e[:T - 5] // (E // 2) == e[:T - 5, :1] // (E // 2)).all())  # one group per token
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        held = step()
    for i in range(3):
        _, x2, _, _, ids2, _ = _problem(T, H, H, r, L, BF, "mixed", 20 + i)
        x.copy_(x2)
        ids.copy_(ids2)
        n.fill_(T - i)
        gr.replay()
        now = step()
        torch.cuda.synchronize()
        for p, q in zip(held, now):
            assert torch.equal(p, q), i


@pytest.mark.parametrize("T", [9, 700, 17000])
def test_lora_output_over_its_input(nv, T):
    """out may be x's memory, also where that is y's; out over b is refused."""
    p = _problem(T, 128, 128, 16, 5, BF, "mixed", 6)
    want = nv.lora_add(*p[:5], scales=p[5])
    x = p[1].clone()
    assert torch.equal(nv.lora_add(p[0], x, *p[2:5], scales=p[5], out=x), want)
    want = nv.lora_add(p[1], *p[1:5], scales=p[5])
    x = p[1].clone()
    assert torch.equal(nv.lora_add(x, x, *p[2:5], scales=p[5], out=x), want)
    L, N, r = p[3].shape
    room = torch.zeros(L * N * r + T * N, dtype=BF, device=DEV)
    room[:L * N * r] = p[3].flatten()
    b, over = room[:L * N * r].view(L, N, r), room[L * N * r - 8 * N:][:T * N].view(T, N)
    with pytest.raises(nv.Nvfp4Error, match="out and b overlap"):
        nv.lora_add(*p[:3], b, p[4], scales=p[5], out=over)


def test_workspaces_are_memory_of_their_own(nv):
    """A workspace counts in bytes, whatever its type; an expanded view, whose
    elements share memory, a short one and one on the host are refused."""
    p = _problem(40, 7168, 64, 16, 3, BF, "one", 0)
    gate = torch.randn(8, 7168, device=DEV).to(BF)
    for call, need in ((lambda ws: nv.lora_add(*p[:5], ws=ws), nv.lora_add_workspace(40, 64, 7168, 16, 3, DEV).numel()),
                       (lambda ws: nv.router_logits(p[1], gate, ws=ws),
                        nv._lib.moe_router_logits_workspace_size(40, 7168, 8, 0))):
        assert need > 256
        want = call(None)
        assert torch.equal(call(torch.empty(need // 4, device=DEV)), want)
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(1, dtype=torch.uint8, device=DEV).expand(need))
        with pytest.raises(ValueError, match="ws must be on"):
            call(torch.empty(need, dtype=torch.uint8))
        with pytest.raises(nv.Nvfp4Error, match="workspace"):
            call(torch.empty(need - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T,L", [(5, 2), (100, 2), (300, 2), (300, 40)])
def test_lora_inner_result_next_to_the_largest_value(nv, T, L, dtype):
    """a x beyond the largest bf16 and still finite: the outputs are finite too."""
    y, x, a, b, ids, _ = _problem(T, 256, 136, 8, L, dtype, "mixed", 13)
    most = torch.finfo(BF).max
    x.zero_()
    x[:, 5], x[:, 200] = most, most / 256  # 1.0039 times the largest bf16: rounds to infinity
    a.zero_()
    a[:, ::2, 5], a[:, ::2, 200] = 1.0, 1.0
    a[:, 1::2, 5], a[:, 1::2, 200] = -1.0, -1.0
    b.mul_(2.0 ** -110)
    b[:, ::3] = 0.0
    ids[T // 2] = L - 1
    out = nv.lora_add(y, x, a, b, ids)
    assert bool(torch.isfinite(out).all())
    _check(out, y, x, a, b, ids, None)


# Outputs so wide and tiles so many that a wave takes several 64-column chunks
# (from 4096 tiles x 256-column blocks on), with whole and ragged last chunks,
# by tiles of 16 tokens (up to 256 tokens and for many adapters) and of 64, and
# every width of r; the last three have one chunk and ranks over 64 in 64-token tiles
WIDE = [(128, 256, 16384, 16, 64), (256, 128, 16392, 40, 5), (256, 64, 8200, 96, 7), (200, 96, 16392, 128, 3),
        (600, 64, 16392, 72, 40), (1000, 64, 16504, 24, 60), (4096, 64, 16392, 32, 8), (4096, 64, 16440, 64, 8),
        (4096, 64, 16392, 72, 8), (2500, 128, 32776, 128, 3), (600, 512, 264, 96, 3), (700, 128, 200, 72, 2),
        (1000, 320, 520, 128, 4)]


@pytest.mark.parametrize("T,K,N,r,L", WIDE)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_lora_wide(nv, T, K, N, r, L, dtype):
    p = _problem(T, K, N, r, L, dtype, "mixed", T + r)
    out = torch.full_like(p[0], 3.0)
    nv.lora_add(*p[:5], scales=p[5], out=out)
    _check(out, *p)
    y = p[0].clone()
    nv.lora_add(y, *p[1:5], scales=p[5], out=y)
    assert torch.equal(y, out)
    p[4].fill_(L - 1)                # one adapter has all tokens
    _check(nv.lora_add(*p[:5], scales=p[5]), *p)
