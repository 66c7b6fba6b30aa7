"""moe_route's refusals (no GPU): every one of them comes before a launch."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _route(nv, logits=FAKE, dtype=1, T=4, E=64, k=8, scoring=0, bias=None, n_group=1, topk_group=1, group_top=1,
           renorm=1, n_tokens=None, ids=FAKE, w=FAKE):
    return nv._lib.moe_route(logits, dtype, T, E, k, scoring, bias, n_group, topk_group, group_top, renorm, 1.0,
                             n_tokens, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(dtype=2), -1), (dict(scoring=2), -1),
    (dict(renorm=2), -1), (dict(E=513), -2), (dict(E=128, k=33), -2), (dict(n_group=0), -1), (dict(n_group=3), -1),
    (dict(topk_group=2), -1), (dict(n_group=8, topk_group=0), -1), (dict(group_top=0), -1), (dict(group_top=3), -1),
    (dict(n_group=16, topk_group=1), -1),  # 8 of 4 experts
    (dict(E=512, n_group=128, topk_group=128), -2), (dict(k=65), -2), (dict(E=4), -1),
    (dict(T=(1 << 27) + 1), -2), (dict(logits=None), -1), (dict(ids=None), -1), (dict(w=None), -1),
    (dict(logits=ctypes.c_void_p(0x10008)), -1), (dict(bias=ctypes.c_void_p(0x10002)), -1),
    (dict(n_tokens=ctypes.c_void_p(0x10001)), -1), (dict(ids=ctypes.c_void_p(0x10002)), -1)])
def test_route_rejects(nv, kw, status):
    assert _route(nv, **kw) == status
    assert b"moe_route" in nv._lib.nvfp4_last_error()


def test_route_empty_batch_is_a_no_op(nv):
    assert _route(nv, logits=None, T=0, ids=None, w=None) == 0


def test_route_binding_rejects_host_tensors(nv):
    with pytest.raises(ValueError, match="GPU"):
        nv.route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        nv.route(torch.zeros(4, 8, dtype=torch.float16), 2)


def _logits(nv, x=FAKE, T=4, H=64, w=FAKE, w_dtype=0, E=8, bias=None, out=FAKE, ws=None, nws=0):
    return nv._lib.moe_router_logits(x, T, H, w, w_dtype, E, bias, out, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(E=0), -1), (dict(w_dtype=2), -1), (dict(H=48), -2), (dict(E=513), -2),
    (dict(H=(1 << 20) + 32), -2), (dict(T=(1 << 26) + 1), -2), (dict(x=None), -1), (dict(w=None), -1),
    (dict(out=None), -1), (dict(x=ctypes.c_void_p(0x10008)), -1), (dict(w=ctypes.c_void_p(0x10004)), -1),
    (dict(out=ctypes.c_void_p(0x10004)), -1), (dict(bias=ctypes.c_void_p(0x10001)), -1)])
def test_router_logits_rejects(nv, kw, status):
    assert _logits(nv, **kw) == status
    assert b"moe_router_logits" in nv._lib.nvfp4_last_error()


def test_router_logits_workspace_and_empty(nv):
    assert _logits(nv, x=None, T=0, w=None, out=None) == 0
    assert nv._lib.moe_router_logits_workspace_size(0, 64, 8, 0) == 0
    for T, H, E, d in ((1, 64, 8, 0), (16384, 7168, 256, 0), (16384, 7168, 256, 1), (5000, 4096, 512, 1)):
        need = nv._lib.moe_router_logits_workspace_size(T, H, E, d)
        if need:
            assert _logits(nv, T=T, H=H, E=E, w_dtype=d, ws=FAKE, nws=need - 1) == -3
            assert b"workspace" in nv._lib.nvfp4_last_error()
            assert _logits(nv, T=T, H=H, E=E, w_dtype=d, ws=ctypes.c_void_p(0x10010), nws=need) == -1


def test_router_logits_binding_rejects_host_tensors(nv):
    with pytest.raises(ValueError, match="GPU"):
        nv.router_logits(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("T,H,E", [(1 << 62, 64, 1 << 62), (1 << 40, 1 << 40, 1 << 40), ((1 << 63) - 1, 64, 8),
                                   (9, 1 << 62, 4), ((1 << 20) + 1, 64, 8), (16, (1 << 20) + 32, 8), (16, 64, 513),
                                   (4096, 48, 8)])
@pytest.mark.parametrize("w_dtype", [0, 1])
def test_router_logits_workspace_of_unsupported_sizes(nv, T, H, E, w_dtype):
    """A size query answers for sizes that a call refuses as well (0: no workspace)."""
    assert nv._lib.moe_router_logits_workspace_size(T, H, E, w_dtype) == 0
    assert _logits(nv, T=T, H=H, E=E, w_dtype=w_dtype) == -2


def _logits_apart(nv, T, w_dtype, H=64, E=8, **over):
    """Operands 4 MiB apart, some of them moved; returns the status."""
    at = {n: (i + 1) << 22 for i, n in enumerate(("x", "w", "bias", "out", "ws"))}
    at.update(over)
    p = {n: ctypes.c_void_p(v) for n, v in at.items()}
    return _logits(nv, p["x"], T, H, p["w"], w_dtype, E, p["bias"], p["out"], p["ws"],
                   nv._lib.moe_router_logits_workspace_size(T, H, E, w_dtype))


@pytest.mark.parametrize("T", [4, 40, 8200])
@pytest.mark.parametrize("w_dtype", [0, 1])
def test_router_logits_refuses_an_output_over_its_inputs(nv, T, w_dtype):
    for name, at, size in (("x", 1 << 22, T * 128), ("w", 2 << 22, 8 * 128 * (1 + w_dtype)), ("bias", 3 << 22, 32)):
        for out in (at, at - T * 32 + 16, at + (size - 1) // 16 * 16):
            assert _logits_apart(nv, T, w_dtype, out=out) == -1
            assert b"logits and %s overlap" % name.encode() in nv._lib.nvfp4_last_error()


def test_router_logits_refuses_a_workspace_over_its_operands(nv):
    T, H, E = 40, 7168, 8                     # slices of K: partial sums in the workspace
    need = nv._lib.moe_router_logits_workspace_size(T, H, E, 0)
    assert need > 0
    for name, at, size in (("x", 1 << 22, T * H * 2), ("w", 2 << 22, E * H * 2), ("bias", 3 << 22, 32),
                           ("logits", 4 << 22, T * E * 4)):
        for ws in (at, at - (need - 1) // 256 * 256, at + (size - 1) // 256 * 256):
            assert _logits_apart(nv, T, 0, H=H, ws=ws) == -1
            assert b"ws and %s overlap" % name.encode() in nv._lib.nvfp4_last_error()


@pytest.mark.parametrize("dtype", [0, 1])
def test_route_refuses_outputs_over_its_operands(nv, dtype):
    T, E, k = 40, 64, 8
    at = {n: (i + 1) << 20 for i, n in enumerate(("logits", "bias", "n_tokens", "ids", "w"))}
    size = {"logits": T * E * (2 + 2 * dtype), "bias": 4 * E, "n_tokens": 4, "ids": 4 * T * k, "w": 4 * T * k}
    for out, name in (("ids", b"ids"), ("w", b"weights")):
        for over in set(at) - {out}:
            for p in (at[over], at[over] - size[out] + 4, at[over] + size[over] - 4):
                now = {n: ctypes.c_void_p(v) for n, v in {**at, out: p}.items()}
                assert _route(nv, T=T, E=E, k=k, dtype=dtype, **now) == -1
                error = nv._lib.nvfp4_last_error()
                assert b"overlap" in error and name in error


def test_router_logits_border_between_slices_and_tiles(nv):
    """The workspace shows which kernel takes a call: above the bound on the
    slices' work (32 x 32 tiles times H) the tiles' partial sums, and for fp32
    weights their three bf16 planes."""
    size = nv._lib.moe_router_logits_workspace_size
    H, E = 1024, 256
    assert size(2048, H, E, 0) == 0 and size(2816, H, E, 1) == 0
    assert size(2049, H, E, 0) == 2 * 2049 * E * 4
    assert size(2817, H, E, 1) == 3 * 2817 * E * 4 + 3 * E * H * 2
    assert size(16387, 512, E, 0) == 0                                        # the kernel stores the result
    assert size(16387, 512, E, 1) == 3 * 16387 * E * 4 + 3 * E * 512 * 2
    # the shapes that test the tiled kernel: all of them have fp32 planes
    for T, H, E in ((16500, 448, 255), (40000, 64, 300), (70001, 576, 4), (4100, 1024, 256), (1100, 7168, 128),
                    (2100, 4096, 101), (3000, 2048, 512), (8191, 320, 260), (5000, 2048, 160), (5001, 2048, 159),
                    (20000, 512, 130), (4500, 2048, 160), (16500, 512, 96)):
        need, planes = size(T, H, E, 1), (3 * E * H * 2 + 255) // 256 * 256
        parts = (need - planes) // (4 * T * E)
        assert parts >= 3 and parts % 3 == 0 and need == planes + (parts * T * E * 4 + 255) // 256 * 256, (T, H, E)


@pytest.mark.parametrize("kw,beyond", [
    (dict(T=1 << 24), dict(T=(1 << 24) + 1)), (dict(E=512), dict(E=513)), (dict(k=32), dict(k=33)),
    (dict(E=512, n_group=64, topk_group=64), dict(E=390, n_group=65, topk_group=65))])
def test_route_limits(nv, kw, beyond):
    """The last supported size reaches the check of the pointers, the next one
    does not."""
    assert _route(nv, logits=None, **kw) == -1
    assert b"null pointer" in nv._lib.nvfp4_last_error()
    assert _route(nv, logits=None, **beyond) == -2


@pytest.mark.parametrize("kw,beyond", [
    (dict(T=1 << 20), dict(T=(1 << 20) + 1)), (dict(E=512), dict(E=513)),
    (dict(H=1 << 20), dict(H=(1 << 20) + 32)), (dict(H=32), dict(H=16))])
def test_router_logits_limits(nv, kw, beyond):
    assert _logits(nv, x=None, **kw) == -1
    assert b"null pointer" in nv._lib.nvfp4_last_error()
    assert _logits(nv, x=None, **beyond) == -2
