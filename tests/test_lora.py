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
