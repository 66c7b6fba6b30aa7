"""Routing of tokens to experts on the GPU against its definition in 64 bits:
the ids are equal, the weights within the tolerance that weight_tolerance derives."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import dev_bf16, dev_f32, host
from router_util import route_rows, weight_tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _check(nv, logits, k, bias=None, scale=1.0, **kw):
    ids, w = nv.route(logits, k, bias=bias, scale=scale, **kw)
    z = host(logits.double())
    want, ww = route_rows(z, k, bias=None if bias is None else host(bias.double()), scale=scale, **kw)
    got, gw = host(ids), host(w).astype(np.float64)
    bad = np.argwhere((got != want).any(1)).ravel()
    assert bad.size == 0, (bad[:5], got[bad[:3]], want[bad[:3]])
    off = np.abs(gw - ww) - weight_tolerance(z, want, ww, scale)
    assert (off <= 0).all(), (off.max(), gw.ravel()[off.argmax()], ww.ravel()[off.argmax()])
    assert (gw[want < 0] == 0).all()
    return ids, w


def _logits(T, E, seed, dtype=torch.float32, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).to(DEV)


def _bias(E, seed):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.round(torch.randn(E, generator=g) * 20) * 0.001).to(DEV)


# (T, E, k, n_group, topk_group, group_top): one lane with one expert up to
# eight (and fifteen: 33 groups of 15 on one lane each), lanes that are not
# filled, experts that do not divide over the lanes
SHAPES = [(1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (5, 8, 2, 1, 1, 1), (1, 256, 8, 1, 1, 1), (7, 63, 4, 1, 1, 1),
          (9, 64, 32, 1, 1, 1), (4, 65, 6, 1, 1, 1), (130, 256, 8, 8, 4, 2), (6, 160, 6, 8, 3, 1),
          (6, 160, 6, 8, 3, 2), (5, 384, 8, 1, 1, 1), (3, 511, 10, 1, 1, 1), (17, 512, 32, 16, 16, 2),
          (4, 495, 12, 33, 20, 2), (4, 128, 2, 64, 1, 2), (5, 12, 3, 3, 2, 2), (2, 510, 9, 51, 7, 1),
          (3, 9, 9, 9, 9, 2), (66, 72, 6, 1, 1, 1)]


@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_top", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_shapes(nv, T, E, k, n_group, topk_group, group_top, scoring, dtype):
    z = _logits(T, E, T * 7 + E + k, dtype)
    for bias in (None, _bias(E, E)):
        for renorm in (True, False):
            _check(nv, z, k, bias=bias, scoring=scoring, n_group=n_group, topk_group=topk_group,
                   group_top=group_top, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_masks_and_extremes(nv, scoring, with_bias, groups):
    E = 32
    z = _logits(16, E, 5)
    lowest = torch.finfo(torch.float32).min
    z[0] = -INF                      # nothing left
    z[1] = NAN                       # nothing left
    z[2] = -INF
    z[2, 17] = -3.0                  # one expert left, fewer than k
    z[3, ::2] = NAN                  # half of them
    z[4] = lowest                    # the lowest value is a value, not a mask
    z[5, :24] = lowest
    z[6, 3] = z[6, 30] = INF         # counts as the largest finite value, twice: they tie
    z[7] = 0.0
    z[7, 1::2] = -0.0                # equal to zero: ties by index
    z[8] = 1.25                      # all equal
    z[9, :8] = -INF                  # a group without a live expert
    z[10] = -200.0                   # scores that vanish in fp32
    z[10, 5] = -199.0
    z[11, :] = torch.linspace(-120, 80, E)
    z[12] = -INF
    z[12, 8:11] = torch.tensor([1.0, 2.0, 3.0])
    z[13, 0] = torch.finfo(torch.float32).max
    z[14] = 1e-40                    # below the normal range
    z[14, 9] = 2e-40
    bias = _bias(E, 3) if with_bias else None
    for renorm in (True, False):
        _check(nv, z, 6, bias=bias, scoring=scoring, n_group=groups[0], topk_group=groups[1], group_top=groups[2],
               renormalize=renorm)
        _check(nv, z.bfloat16(), 6, bias=bias, scoring=scoring, n_group=groups[0], topk_group=groups[1],
               group_top=groups[2], renormalize=renorm)


def test_route_bias_switches_experts_off_and_on(nv):
    z = _logits(20, 48, 9)
    b = _bias(48, 9)
    b[3], b[20], b[21] = NAN, -INF, -INF
    b[40], b[7] = INF, INF           # always first, by index
    ids, _ = _check(nv, z, 5, bias=b, scoring="sigmoid")
    assert not np.isin(host(ids), [3, 20, 21]).any()
    assert (host(ids)[:, :2] == [7, 40]).all()
    b = torch.full((48,), -INF, device=DEV)
    b[11] = 0.5
    ids, w = _check(nv, z, 5, bias=b, scoring="softmax")
    assert (host(ids)[:, 1:] == -1).all() and (host(w)[:, 1:] == 0).all()
    b[:] = 1e30                      # a bias that swallows every score: fp64 does not separate them either
    ids, _ = nv.route(z, 5, bias=b)
    assert (host(ids) == np.arange(5)).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2)])
def test_route_decides_between_neighbours(nv, scoring, groups):
    """Choices that lie closer together than fp32 scores are exact."""
    E, T = 64, 64
    z = _logits(T, E, 21, std=0.5)
    zz = z.double()
    s = torch.softmax(zz, 1) if scoring == "softmax" else torch.sigmoid(zz)
    # one bias vector per row: every expert's choice lands next to 0.75, the
    # rounding of the bias to fp32 decides
    for t in range(T):
        b = (0.75 - s[t]).float()
        _check(nv, z[t:t + 1], 8, bias=b, scoring=scoring, n_group=groups[0], topk_group=groups[1],
               group_top=groups[2])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_decides_between_neighbouring_groups(nv, scoring):
    """Groups whose sums differ below fp32's resolution, without a bias."""
    E, G = 64, 8
    z = _logits(G, E, 33)
    for t in range(G):
        g = torch.Generator().manual_seed(t)
        base = torch.randn(E // G, generator=g)
        for j in range(G):           # the same values in another order, one of them a step away
            v = base[torch.randperm(E // G, generator=g)].clone()
            v[v.argmax()] = torch.nextafter(v.max(), torch.tensor(INF if j % 3 else -INF))
            z[t, j * (E // G):(j + 1) * (E // G)] = v.to(DEV)
    _check(nv, z, 8, scoring=scoring, n_group=G, topk_group=4, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_groups_with_large_opposite_biases(nv, scoring):
    """A group's value may be small where its terms are large: what their
    roundings leave decides then, not the sum's size."""
    E, G = 64, 8
    z = _logits(40, E, 12)
    b = torch.full((E,), -INF, device=DEV)
    for g in range(G):               # two experts a group, 1e6 up and down: fp32 sums lose the scores
        b[8 * g + g], b[8 * g + (g + 3) % 8] = 1.0e6, -1.0e6
    _check(nv, z, 2, bias=b, scoring=scoring, n_group=G, topk_group=3, group_top=2)
    b = torch.where(b > 0, b - 0.75, b)
    _check(nv, z, 4, bias=b, scoring=scoring, n_group=G, topk_group=2, group_top=2)


def test_route_large_batch(nv):
    """Many tokens, against torch in 64 bits (values without ties)."""
    T, E, k = 40001, 256, 8
    z = _logits(T, E, 2)
    b = _bias(E, 2)
    ids, w = nv.route(z, k, scoring="sigmoid", bias=b)
    s = torch.sigmoid(z.double())
    c, want = torch.sort(s + b.double(), dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want[:, :k])
    part = s.gather(1, want[:, :k])
    part = part / part.sum(1, keepdim=True)
    assert float((w - part).abs().max()) <= 40 * 2.0 ** -24


def test_route_padded_batch_and_out(nv):
    T, E, k = 37, 96, 4
    z = _logits(T, E, 4)
    ids0, w0 = nv.route(z, k)
    for n in (0, 1, 36, 37, 50, -3):
        out = (torch.full((T, k), 77, dtype=torch.int32, device=DEV), torch.full((T, k), 7.0, device=DEV))
        ids, w = nv.route(z, k, n_tokens=torch.tensor([n], dtype=torch.int32, device=DEV), out=out)
        assert ids is out[0] and w is out[1]
        m = max(0, min(n, T))
        assert torch.equal(ids[:m], ids0[:m]) and torch.equal(w[:m], w0[:m])
        assert (ids[m:] == -1).all() and (w[m:] == 0).all()


def test_route_graph_and_streams(nv):
    """A captured call follows its inputs over replays, with eager calls on
    the same stream and another one in between."""
    T, E, k = 50, 160, 6
    z, b = _logits(T, E, 6), _bias(E, 6)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    kw = dict(scoring="sigmoid", bias=b, n_group=8, topk_group=3, group_top=2, n_tokens=n)
    nv.route(z, k, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, w = nv.route(z, k, **kw)
    side = torch.cuda.Stream()
    for i in range(4):
        z.copy_(_logits(T, E, 60 + i))
        n.fill_(T - 11 * i)
        g.replay()
        eager = nv.route(z, k, **kw)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = nv.route(z, k, **kw)
        torch.cuda.synchronize()
        for a in (eager, other):
            assert torch.equal(a[0], ids) and torch.equal(a[1], w), i


def test_route_refuses_bad_tensors(nv):
    z = _logits(8, 32, 1)
    for bad in (dict(bias=torch.zeros(31, device=DEV)), dict(bias=torch.zeros(32, device=DEV).bfloat16()),
                dict(scoring="tanh"), dict(n_tokens=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(n_tokens=torch.zeros(1, dtype=torch.int32)),
                dict(out=(torch.zeros(8, 3, dtype=torch.int32, device=DEV), torch.zeros(8, 4, device=DEV)))):
        with pytest.raises(ValueError):
            nv.route(z, 4, **bad)
    with pytest.raises(ValueError, match="contiguous"):
        nv.route(z[:, ::2], 4)
    with pytest.raises(nv.Nvfp4Error):
        nv.route(z, 33)
    with pytest.raises(nv.Nvfp4Error):
        nv.route(z, 0)
    ids, w = nv.route(z[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_route_feeds_the_expert_ffn(nv):
    """Routing and experts together: the ids and weights go into the expert FFN as
    they are; a token with every expert masked gets a zero row."""
    cfg = synth.TINY
    x = dev_bf16(synth.activations(cfg))
    w = [synth.expert_weights(cfg, e, device=DEV) for e in range(cfg.E)]
    w1 = nv.quantize_experts(torch.stack([a for a, _ in w]))
    w2 = nv.quantize_experts(torch.stack([b for _, b in w]))
    z = _logits(cfg.T, cfg.E, 8)
    z[5] = -INF
    z[9, 1:] = -INF
    ids, wt = _check(nv, z, cfg.topk)
    a2 = dev_f32(cfg.a2_gs)
    y = nv.moe_expert_ffn(x, ids, wt, *w1, *w2, a2, out_dtype=torch.float32)
    want, ww = route_rows(host(z.double()), cfg.topk)
    y2 = nv.moe_expert_ffn(x, torch.from_numpy(want).to(DEV), torch.from_numpy(ww.astype(np.float32)).to(DEV), *w1,
                           *w2, a2, out_dtype=torch.float32)
    assert (y[5] == 0).all() and (y[9] != 0).any()
    # the weights differ by roundings only, and the FFN is linear in them
    assert float((y - y2).norm() / y2.norm()) <= 64 * 2.0 ** -24


def test_route_orders_by_what_64_bits_hold(nv):
    """With a bias, scores that are one value in 64 bits tie and go by index;
    one step before that the larger logit is first; without a bias the logits
    decide throughout."""
    bias = torch.zeros(4, device=DEV)
    for scoring, apart, same in (("sigmoid", [34.0, 34.5, 33.0, -1.0], [40.0, 41.0, 60.0, -1.0]),
                                 ("softmax", [-700.0, -699.0, -701.0, 0.0], [-800.0, -799.0, -801.0, 0.0])):
        z = torch.tensor([apart, same], device=DEV)
        ids, _ = _check(nv, z, 4, bias=bias, scoring=scoring)
        first = 1 if scoring == "softmax" else 0
        assert host(ids)[:, first:first + 3].tolist() == [[1, 0, 2], [0, 1, 2]]
        ids, _ = _check(nv, z, 4, scoring=scoring)
        assert host(ids)[:, first:first + 3].tolist() == [[1, 0, 2], [2, 1, 0] if scoring == "sigmoid" else [1, 0, 2]]
    # group sums without a bias: 1 + 1 in both, then in the logits' order inside the group that stays
    z = torch.tensor([[40.0, 41.0, 50.0, 51.0], [33.0, 34.0, 50.0, 51.0]], device=DEV)
    ids, _ = _check(nv, z, 2, scoring="sigmoid", n_group=2, topk_group=1, group_top=2)
    assert host(ids).tolist() == [[1, 0], [3, 2]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group", [(256, 1), (512, 1), (510, 3), (510, 5), (504, 9), (510, 17), (495, 33)])
@pytest.mark.parametrize("std", [0.02, 2.0])
def test_route_small_gaps_with_every_lane_layout(nv, scoring, E, n_group, std):
    """One to fifteen experts per lane, flat and peaked scores, biases that
    bring the choices of neighbours to within a few roundings of fp32."""
    z = _logits(24, E, E + n_group, std=std)
    z[:, 3] += 4.0                   # with a score next to 1 the sum's error weighs most
    s = torch.softmax(z.double(), 1) if scoring == "softmax" else torch.sigmoid(z.double())
    g = torch.Generator().manual_seed(E)
    step = torch.randint(-40, 41, (E,), generator=g).to(DEV).double() * 2.0 ** -25
    for t in range(0, 24, 3):
        bias = (0.5 - s[t] + step).float()
        _check(nv, z[t:t + 1].clone(), 8, bias=bias, scoring=scoring, n_group=n_group, topk_group=max(1, n_group // 2),
               group_top=2 if n_group > 1 else 1)


# ------------------------------------------------------------------ gate projection
def _gate(T, H, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).bfloat16()
    w = (torch.randn(E, H, generator=g) * 0.02).to(dtype)
    return x.to(DEV), w.to(DEV), (torch.randn(E, generator=g) * 0.1).to(DEV)


def _gate_check(y, x, w, bias):
    """Products are exact, so only the fp32 accumulation errs: at most H + 64
    roundings of partial sums, none larger than the sum of the terms'
    magnitudes; and over all elements like a walk of H / 8 + 20 steps (eight
    or more products enter a sum at once, and the slices' sums are added),
    each uniform within half a step of a partial sum (variance a third of its
    square), allowed twice.  The terms are independent with mean zero, so a
    partial sum of them has at most the mean square of the whole, which is the
    sum of the terms' squares (the result itself may be smaller by cancellation
    and says nothing about the sums on the way)."""
    H = x.shape[1]
    xd, wd = x.double(), w.double()
    want, size = xd @ wd.t().contiguous(), xd.abs() @ wd.abs().t().contiguous()
    square = xd.square() @ wd.square().t().contiguous()
    if bias is not None:
        want, size, square = want + bias.double(), size + bias.double().abs(), square + bias.double().square()
    err = (y.double() - want).abs()
    assert bool((err <= size * (H + 64) * 2.0 ** -24).all())
    rel = float(err.norm() / square.sum().sqrt())
    assert rel <= 2 * ((H / 8 + 20) / 3) ** 0.5 * 2.0 ** -24, rel


GATE_SHAPES = [(1, 32, 1), (1, 7168, 256), (3, 64, 5), (16, 256, 8), (17, 96, 17), (33, 1280, 160), (100, 512, 511),
               (129, 2048, 72), (130, 7168, 256), (300, 160, 512), (1000, 768, 40), (513, 1024, 128),
               (2049, 480, 200), (4100, 256, 256), (8, 2048, 33), (9, 2048, 33), (256, 640, 511), (257, 640, 512),
               (16, 7168, 8), (700, 4096, 72), (2000, 4096, 130)]


@pytest.mark.parametrize("T,H,E", GATE_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router_logits_shapes(nv, T, H, E, dtype):
    x, w, b = _gate(T, H, E, dtype, T + H + E)
    _gate_check(nv.router_logits(x, w), x, w, None)
    out = torch.full((T, E), 9.0, device=DEV)
    y = nv.router_logits(x, w, bias=b, out=out)
    assert y is out
    _gate_check(y, x, w, b)


@pytest.mark.parametrize("T", [3, 700, 5000])
def test_router_logits_uses_all_bits_of_a_32_bit_weight(nv, T):
    """Differences of neighbouring weights: only the last bits are left, and
    the answer is exact."""
    H, E = 256, 40
    w = torch.zeros(E, H, device=DEV)
    g = torch.Generator().manual_seed(0)
    v = (torch.rand(E, H // 2, generator=g) + 1.0).to(DEV)
    nxt = torch.nextafter(v, torch.full_like(v, 2.0))
    col = torch.arange(E, device=DEV)
    w[col, 2 * col] = v[col, col]
    w[col, 2 * col + 1] = nxt[col, col]
    x = torch.zeros(T, H, device=DEV)
    x[:, 0::2], x[:, 1::2] = -1.0, 1.0
    y = nv.router_logits(x.bfloat16(), w)
    assert torch.equal(y, (nxt - v)[col, col].expand(T, E))


@pytest.mark.parametrize("T", [5, 600, 4500])
def test_router_logits_rows_are_independent(nv, T):
    """A token with NaN or infinite activations spoils its own row only."""
    x, w, _ = _gate(T, 512, 96, torch.bfloat16, 3)
    y0 = nv.router_logits(x, w)
    x2 = x.clone()
    x2[1], x2[T - 1, 7] = NAN, INF
    y = nv.router_logits(x2, w)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1] = keep[T - 1] = False
    assert torch.equal(y[keep], y0[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[T - 1]).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [7, 5000])
def test_router_logits_graph_with_routing(nv, T, dtype):
    """Projection and routing captured together, replayed on new inputs."""
    x, w, b = _gate(T, 384, 64, dtype, 4)
    nv.route(nv.router_logits(x, w, bias=b), 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = nv.router_logits(x, w, bias=b)
        ids, wt = nv.route(y, 4)
    for i in range(3):
        x.copy_(_gate(T, 384, 64, dtype, 40 + i)[0])
        g.replay()
        y2 = nv.router_logits(x, w, bias=b)
        i2, w2 = nv.route(y2, 4)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(ids, i2) and torch.equal(wt, w2), i


def test_router_logits_refuses_bad_tensors(nv):
    x, w, b = _gate(4, 64, 8, torch.bfloat16, 1)
    for args, kw in (((x, w[:, :32].contiguous()), {}), ((x, w.half()), {}), ((x.float(), w), {}),
                     ((x, w), dict(bias=b[:7])), ((x, w), dict(out=torch.empty(4, 7, device=DEV))),
                     ((x.t(), w), {}), ((x, w.cpu()), {}), ((x, w), dict(bias=b.double()))):
        with pytest.raises(ValueError):
            nv.router_logits(*args, **kw)
    with pytest.raises(nv.Nvfp4Error):
        nv.router_logits(x[:, :48].contiguous(), w[:, :48].contiguous())
    assert nv.router_logits(x[:0], w).shape == (0, 8)


# Sizes beyond the sliced kernel's range for both weight types, which the tiled
# kernel takes: one K step and odd numbers of them, a last tile of few tokens,
# one part (the bias and the store in the kernel itself) and several, whole and
# cut register quads of experts, more experts than one tile, few of them; the
# first sizes on either side of the border between the kernels
TILE_SHAPES = [(16387, 512, 256), (16500, 448, 255), (40000, 64, 300), (70001, 576, 4), (4100, 1024, 256),
               (1100, 7168, 128), (2100, 4096, 101), (3000, 2048, 512), (8191, 320, 260), (2048, 1024, 256),
               (2049, 1024, 256), (2816, 1024, 256), (2817, 1024, 256)]


@pytest.mark.parametrize("T,H,E", TILE_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router_logits_tiles(nv, T, H, E, dtype):
    x, w, b = _gate(T, H, E, dtype, T + H + E)
    _gate_check(nv.router_logits(x, w), x, w, None)
    room = torch.full((T * E + 8,), 9.0, device=DEV)
    y = nv.router_logits(x, w, bias=b, out=room[:T * E].view(T, E))
    _gate_check(y, x, w, b)
    assert bool((room[T * E:] == 9.0).all())


@pytest.mark.parametrize("T,H,E", [(5000, 2048, 160), (5001, 2048, 159), (20000, 512, 130)])
def test_router_logits_tiles_use_all_bits_of_a_32_bit_weight(nv, T, H, E):
    w = torch.zeros(E, H, device=DEV)
    g = torch.Generator().manual_seed(1)
    v = (torch.rand(E, generator=g) + 1.0).to(DEV)
    nxt = torch.nextafter(v, torch.full_like(v, 2.0))
    e = torch.arange(E, device=DEV)
    w[e, 3 * e], w[e, 3 * e + 1] = v, nxt
    x = torch.zeros(T, H, device=DEV)
    x[:, 0::3], x[:, 1::3] = -1.0, 1.0  # of an expert's two weights, whatever else lies there is zero
    y = nv.router_logits(x.bfloat16(), w)
    assert torch.equal(y, (nxt - v).expand(T, E))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,E", [(4500, 2048, 160), (16500, 512, 96)])
def test_router_logits_tile_rows_are_independent(nv, T, H, E, dtype):
    x, w, _ = _gate(T, H, E, dtype, 3)
    y0 = nv.router_logits(x, w)
    x2 = x.clone()
    x2[1], x2[T - 1, 7], x2[130, H - 1] = NAN, INF, -INF
    y = nv.router_logits(x2, w)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[1, 130, T - 1]] = False
    assert torch.equal(y[keep], y0[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[[130, T - 1]]).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,E", [(5000, 2048, 160), (16500, 512, 96)])
def test_router_logits_tiles_in_a_graph(nv, T, H, E, dtype):
    """Projection and routing captured together, replayed on new inputs and
    weights, with eager calls between the replays and on another stream."""
    x, w, b = _gate(T, H, E, dtype, 4)
    nv.route(nv.router_logits(x, w, bias=b), 4)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        y = nv.router_logits(x, w, bias=b)
        ids, wt = nv.route(y, 4)
    for i in range(3):
        for dst, src in zip((x, w, b), _gate(T, H, E, dtype, 40 + i)):
            dst.copy_(src)
        g.replay()
        y2 = nv.router_logits(x, w, bias=b)
        i2, wt2 = nv.route(y2, 4)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y3 = nv.router_logits(x, w, bias=b)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(y, y3) and torch.equal(ids, i2) and torch.equal(wt, wt2), i
