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
