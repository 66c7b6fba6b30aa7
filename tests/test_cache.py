"""The cache calls' refusals (no GPU): every one of them comes before a launch."""
import ctypes

import numpy as np
import pytest
import torch

from block_util import E4M3, to_mxfp8, values

AT = dict(rows=0x10000000, q=0x20000000, s=0x30000000, gs=0x40000000, slots=0x50000000, pages=0x60000000,
          cu=0x70000000)


@pytest.fixture(scope="module")
def nv():
    import quantization_nvfp4_quantize_amd as nv
    return nv


def _parts(nv, n, **over):
    parts = (nv.CachePart * 2)()
    for i in range(2):
        for f, v in dict(rows=AT["rows"], row_stride=64, R=64, q=AT["q"], s=AT["s"], gs=AT["gs"]).items():
            setattr(parts[i], f, v + (i << 24) if f in ("rows", "q", "s") else v)
    for f, v in over.items():
        setattr(parts[n - 1], f, v)
    return parts


def _call(nv, which, format=0, n=1, T=4, slots=AT["slots"], n_slots=16, dtype=0, pages=AT["pages"], B=2, wide=3,
          page=4, cu=AT["cu"], null=False, **part):
    p, lib = None if null else _parts(nv, n, **part), nv._lib
    if which == "write":
        return lib.kv_cache_write(format, p, n, T, slots, n_slots, None)
    if which == "read":
        return lib.kv_cache_read(format, p, n, T, slots, n_slots, dtype, None)
    return lib.kv_cache_read_pages(format, p, n, T, pages, B, wide, page, cu, n_slots, dtype, None)


COMMON = [(dict(format=3), -1), (dict(format=-1), -1), (dict(n=0), -1), (dict(n=3), -1), (dict(T=-1), -1),
          (dict(n_slots=-1), -1), (dict(n_slots=1 << 31), -2), (dict(null=True), -1), (dict(R=0), -1), (dict(R=24), -1),
          (dict(format=1, R=48, row_stride=48), -1), (dict(format=2, R=16, row_stride=16), -1),
          (dict(R=(1 << 20) + 32, row_stride=(1 << 20) + 32), -2), (dict(T=1 << 28), -2), (dict(rows=None), -1),
          (dict(q=None), -1), (dict(s=None), -1), (dict(gs=None), -1), (dict(rows=AT["rows"] + 8), -1),
          (dict(q=AT["q"] + 8), -1), (dict(gs=AT["gs"] + 2), -1), (dict(n=2, q=None), -1), (dict(n=2, R=40), -1)]


@pytest.mark.parametrize("which", ["write", "read", "read_pages"])
@pytest.mark.parametrize("kw,status", COMMON)
def test_cache_rejects(nv, which, kw, status):
    assert _call(nv, which, **kw) == status
    assert b"kv_cache_" + which.encode() in nv._lib.nvfp4_last_error()


@pytest.mark.parametrize("which,kw,status", [
    ("write", dict(row_stride=60), -1), ("write", dict(row_stride=56), -1), ("write", dict(slots=None), -1),
    ("write", dict(slots=AT["slots"] + 2), -1), ("read", dict(slots=None), -1), ("read", dict(dtype=2), -1),
    ("read_pages", dict(dtype=-1), -1), ("read_pages", dict(B=-1), -1), ("read_pages", dict(wide=-1), -1),
    ("read_pages", dict(page=0), -1), ("read_pages", dict(pages=None), -1), ("read_pages", dict(cu=None), -1),
    ("read_pages", dict(cu=AT["cu"] + 2), -1), ("read_pages", dict(B=(1 << 31) - 1), -2),
    ("read_pages", dict(page=1 << 31), -2)])
def test_cache_rejects_its_own(nv, which, kw, status):
    assert _call(nv, which, **kw) == status


@pytest.mark.parametrize("which,kw", [
    ("write", dict(q=AT["rows"] + 64)), ("write", dict(s=AT["rows"] + 511)), ("write", dict(s=AT["q"] + 511)),
    ("write", dict(q=AT["slots"])), ("write", dict(s=AT["gs"])), ("write", dict(n=2, q=AT["q"] + 496)),
    ("read", dict(rows=AT["q"] + 496)), ("read", dict(rows=AT["s"] + 48)), ("read", dict(rows=AT["slots"])),
    ("read", dict(n=2, rows=AT["rows"] + 496)), ("read", dict(rows=AT["gs"])),
    ("read_pages", dict(rows=AT["pages"] + 16)), ("read_pages", dict(rows=AT["cu"]))])
def test_cache_refuses_to_write_over_operands(nv, which, kw):
    assert _call(nv, which, **kw) == -1
    assert b"overlap" in nv._lib.nvfp4_last_error()


def test_cache_nothing_to_do(nv):
    none = dict(rows=None, q=None, s=None, gs=None)
    assert _call(nv, "write", T=0, slots=None, **none) == 0
    assert _call(nv, "write", n_slots=0) == 0
    assert _call(nv, "read", T=0, slots=None, **none) == 0
    assert _call(nv, "read_pages", T=0, pages=None, cu=None, **none) == 0
    assert _call(nv, "read_pages", B=0, pages=None, cu=None) == 0


def test_cache_binding_rejects(nv):
    q, s = torch.zeros(4, 2, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, dtype=torch.uint8)
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        nv.cache_write(x, slots, (q, s))
    with pytest.raises(ValueError, match="GPU"):
        nv.cache_read((q, s), slots)
    with pytest.raises(ValueError, match="GPU"):
        nv.cache_read_pages((q, s), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4, 3)
    with pytest.raises(ValueError, match="format"):
        nv.cache_empty(4, (2, 64), format="int4", device="cpu")
    with pytest.raises(ValueError, match="multiple"):
        nv.cache_empty(4, (2, 48), device="cpu")
    with pytest.raises(ValueError, match="global scale"):
        nv.cache_empty(4, (2, 48), format="nvfp4", device="cpu")
    with pytest.raises(ValueError, match="global scale"):
        nv.cache_empty(4, (2, 64), device="cpu", gs=torch.ones(1))
    assert [t.shape[-1] for t in nv.cache_empty(4, (2, 64), device="cpu")] == [64, 2]
    assert [t.shape[-1] for t in nv.cache_empty(4, (64,), "nvfp4", "cpu", torch.ones(1))] == [32, 4, 1]


def test_mxfp8_reference_against_definitions():
    """The reference's own rounding: every code's own value stays, the block's
    maximum never saturates, the scale is the smallest, errors are at most half
    a step."""
    assert E4M3[0x7e] == 448 and E4M3[1] == 2.0 ** -9 and np.isnan(E4M3[127])
    for top in (448.0, 449.0, 224.0, 1.75, 1.7500001, 1.0, 2.0 ** -130, 0.0, 3e38):
        x = np.zeros((1, 32))
        x[0, 0], x[0, 1] = top, -top / 3
        q, c = to_mxfp8(x)
        scale = 2.0 ** (int(c[0, 0]) - 127)
        assert top <= 448 * scale and (c[0, 0] == 0 or top > 448 * scale / 2)
        err = np.abs(values(q, c, "mxfp8") - x)
        assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)).all()
    grid = np.concatenate([E4M3[:127], np.zeros(31 * 5 - 127)]).reshape(5, 31)
    q, c = to_mxfp8(np.concatenate([np.full((5, 1), 448.0), grid], axis=1))  # 448 in every block: code 127
    assert (c == 127).all() and (q[:, 0] == 0x7e).all() and (q[:, 1:].ravel()[:127] == np.arange(127)).all()
