"""nvfp4_matvec's and mxfp4_matvec's refusals (no GPU): every one of them comes before a launch."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000000)  # never dereferenced: validation fails first
FAR = ctypes.c_void_p(0x90000000)


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _nvfp4(nv, x=FAKE, M=2, K=64, q=FAKE, s=FAKE, gs=FAKE, N=33, dtype=0, out=FAR):
    return nv._lib.nvfp4_matvec(x, M, K, q, s, gs, N, dtype, out, None)


def _mxfp4(nv, x=FAKE, M=2, K=64, q=FAKE, s=FAKE, N=33, dtype=0, out=FAR):
    return nv._lib.mxfp4_matvec(x, M, K, q, s, N, dtype, out, None)


BAD = [(dict(M=-1), -1), (dict(K=0), -1), (dict(N=0), -1), (dict(dtype=2), -1), (dict(K=48), -2), (dict(K=16), -2),
       (dict(M=(1 << 20) + 1), -2), (dict(K=(1 << 20) + 32), -2), (dict(N=(1 << 20) + 1), -2), (dict(x=None), -1),
       (dict(q=None), -1), (dict(s=None), -1), (dict(out=None), -1), (dict(x=ctypes.c_void_p(0x10000008)), -1),
       (dict(q=ctypes.c_void_p(0x10000008)), -1), (dict(s=ctypes.c_void_p(0x10000002)), -1),
       (dict(out=ctypes.c_void_p(0x90000008)), -1), (dict(out=FAKE), -1)]


@pytest.mark.parametrize("kw,status", BAD + [(dict(gs=None), -1), (dict(gs=ctypes.c_void_p(0x10000002)), -1)])
def test_nvfp4_matvec_rejects(nv, kw, status):
    assert _nvfp4(nv, **kw) == status
    assert b"nvfp4_matvec" in nv._lib.nvfp4_last_error()


@pytest.mark.parametrize("kw,status", BAD)
def test_mxfp4_matvec_rejects(nv, kw, status):
    assert _mxfp4(nv, **kw) == status
    assert b"mxfp4_matvec" in nv._lib.nvfp4_last_error()


def test_matvec_without_tokens_needs_nothing(nv):
    assert _nvfp4(nv, M=0, x=None, q=None, s=None, gs=None, out=None) == 0
    assert _mxfp4(nv, M=0, x=None, q=None, s=None, out=None) == 0


# M 2, K 64, N 33: out has 132 bytes
@pytest.mark.parametrize("name,size", [("x", 256), ("q", 33 * 32), ("s", 33 * 4), ("gs", 4)])
def test_matvec_refuses_an_output_over_what_it_reads(nv, name, size):
    at = 0x20000000
    for out in (at, at - 128, at + (size - 1) // 16 * 16):
        assert _nvfp4(nv, out=ctypes.c_void_p(out), **{name: ctypes.c_void_p(at)}) == -1
        assert b"overlap" in nv._lib.nvfp4_last_error()


def test_matvec_binding_rejects(nv):
    x, q, s = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), None
    with pytest.raises(ValueError, match="GPU"):
        nv.matvec(x, q, torch.zeros(8, 4, dtype=torch.uint8), torch.ones(1))
    with pytest.raises(ValueError, match="GPU"):
        nv.mx_matvec(x, q, torch.zeros(8, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="x must be"):
        nv.mx_matvec(x[0], q, s)
