"""nvfp4_lora_add's refusals (no GPU): every one of them comes before a launch."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
FAR = ctypes.c_void_p(0x10000000)


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _add(nv, y=FAKE, dtype=0, T=4, N=64, x=FAKE, K=64, a=FAKE, b=FAKE, r=8, L=2, ids=FAKE, scales=None, out=FAR,
         ws=FAKE, nws=1 << 30):
    return nv._lib.nvfp4_lora_add(y, dtype, T, N, x, K, a, b, r, L, ids, scales, out, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(r=0), -1), (dict(L=0), -1), (dict(dtype=2), -1),
    (dict(K=48), -2), (dict(N=60), -2), (dict(r=12), -2), (dict(r=136), -2), (dict(L=513), -2),
    (dict(T=(1 << 20) + 1), -2), (dict(K=(1 << 20) + 32), -2), (dict(N=(1 << 20) + 8), -2),
    (dict(y=None), -1), (dict(x=None), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(ids=None), -1),
    (dict(out=None), -1), (dict(y=ctypes.c_void_p(0x10008)), -1), (dict(x=ctypes.c_void_p(0x10002)), -1),
    (dict(a=ctypes.c_void_p(0x10008)), -1), (dict(b=ctypes.c_void_p(0x10008)), -1),
    (dict(out=ctypes.c_void_p(0x10000008)), -1), (dict(ids=ctypes.c_void_p(0x10002)), -1),
    (dict(scales=ctypes.c_void_p(0x10002)), -1), (dict(ws=None), -3), (dict(ws=ctypes.c_void_p(0x10010)), -1),
    (dict(out=ctypes.c_void_p(0x10000 + 256)), -1)])
def test_lora_rejects(nv, kw, status):
    assert _add(nv, **kw) == status
    assert b"nvfp4_lora_add" in nv._lib.nvfp4_last_error()


def test_lora_overlap_counts_bytes(nv):
    at = 4 * 64 * 2
    assert _add(nv, out=ctypes.c_void_p(0x10000 + at - 16)) == -1
    assert b"overlap" in nv._lib.nvfp4_last_error()
    assert _add(nv, dtype=1, out=ctypes.c_void_p(0x10000 + at)) == -1
    assert b"overlap" in nv._lib.nvfp4_last_error()


def test_lora_workspace_and_empty(nv):
    size = nv._lib.nvfp4_lora_add_workspace_size
    assert _add(nv, y=None, T=0, x=None, a=None, b=None, ids=None, out=None, ws=None, nws=0) == 0
    assert size(0, 64, 64, 8, 2) == 0 and size(4, 64, 48, 8, 2) == 0
    for T, L in ((1, 1), (16, 500), (1024, 3), (1025, 512), (100000, 512)):
        need = size(T, 64, 64, 32, L)
        assert need >= T * 32 * 4
        assert _add(nv, T=T, L=L, r=32, nws=need - 1) == -3
        assert b"workspace" in nv._lib.nvfp4_last_error()


def test_lora_binding_rejects_host_tensors(nv):
    h = torch.bfloat16
    with pytest.raises(ValueError, match="GPU"):
        nv.lora_add(torch.zeros(4, 64, dtype=h), torch.zeros(4, 32, dtype=h), torch.zeros(2, 8, 32, dtype=h),
                    torch.zeros(2, 64, 8, dtype=h), torch.zeros(4, dtype=torch.int32))


def _apart(nv, T=4, N=64, K=64, r=8, L=2, **over):
    """Operands 1 MiB apart (16 KiB and less each), some of them moved."""
    at = {n: (i + 1) << 20 for i, n in enumerate(("y", "x", "a", "b", "ids", "scales", "out", "ws"))}
    at.update(over)
    need = nv._lib.nvfp4_lora_add_workspace_size(T, N, K, r, L)
    p = {n: ctypes.c_void_p(v) for n, v in at.items()}
    return nv._lib.nvfp4_lora_add(p["y"], 0, T, N, p["x"], K, p["a"], p["b"], r, L, p["ids"], p["scales"], p["out"],
                                  p["ws"], need, None)


# bytes of a, b, ids, scales for T 4, N 64, K 64, r 8, L 2; out has 512
@pytest.mark.parametrize("name,at,size", [("a", 3 << 20, 2048), ("b", 4 << 20, 2048), ("ids", 5 << 20, 16),
                                          ("scales", 6 << 20, 8)])
def test_lora_refuses_an_output_over_what_it_reads(nv, name, at, size):
    for out in (at, at - 512 + 16, at + (size - 1) // 16 * 16):
        assert _apart(nv, out=out) == -1
        assert b"out and %s overlap" % name.encode() in nv._lib.nvfp4_last_error()


@pytest.mark.parametrize("name,at,size", [("y", 1 << 20, 512), ("x", 2 << 20, 512), ("a", 3 << 20, 2048),
                                          ("b", 4 << 20, 2048), ("ids", 5 << 20, 16), ("scales", 6 << 20, 8),
                                          ("out", 7 << 20, 512)])
def test_lora_refuses_a_workspace_over_its_operands(nv, name, at, size):
    need = nv._lib.nvfp4_lora_add_workspace_size(4, 64, 64, 8, 2)
    for ws in (at, at - (need - 1) // 256 * 256, at + (size - 1) // 256 * 256):
        assert _apart(nv, ws=ws) == -1
        assert b"ws and %s overlap" % name.encode() in nv._lib.nvfp4_last_error()
