"""Pointers that no load or store of their type may start at, refused by the
row products before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

FAKE, BIG = 0x1000, 1 << 30
R = ctypes.byref


@pytest.fixture(scope="module")
def tq():
    from group_scale_search_b200 import build
    build.build()
    import group_scale_search_b200 as g
    g.lib()
    return g


def records(tq, fmt, **kw):
    a = dict(packed=FAKE, scales=FAKE, zeros=FAKE if fmt in tq._INT4 else None, glob=FAKE if fmt == tq.NVFP4_G16 else None)
    a.update(kw)
    return tq._Records(a["packed"], a["scales"], a["zeros"], a["glob"], fmt, 0, 1, 64, 128)


def refused(tq, status):
    return status == 1 and b"aligned" in tq.lib().tq_last_error_string()


@pytest.mark.parametrize("at", [0x1001, 0x1002, 0x1003])
def test_global_scales(tq, at):
    L, x, d = tq.lib(), tq._Mat(FAKE, 1, 0, 1, 40, 128, 128, 0), tq._Mat(FAKE, 1, 0, 1, 40, 64, 64, 0)
    w, good = records(tq, tq.NVFP4_G16, glob=at), records(tq, tq.NVFP4_G16)
    assert refused(tq, L.tq_dequant_matmul(R(w), R(x), None, FAKE, 1, 64, FAKE, BIG, None))
    assert refused(tq, L.tq_dequant_matmul_backward(R(w), R(d), None, FAKE, 128, FAKE, BIG, None))
    assert refused(tq, L.tq_gated_ffn(R(good), R(w), 0, R(x), None, FAKE, 1, 64, FAKE, BIG, None))
    assert refused(tq, L.tq_gated_ffn_backward(R(w), R(good), 0, R(x), R(d), None, FAKE, 128, FAKE, BIG, None))
    assert refused(tq, L.tq_head_loss(R(w), R(x), FAKE, FAKE, FAKE, FAKE, BIG, None))


@pytest.mark.parametrize("at", [0x1001, 0x1002, 0x1003])
def test_loss_vectors(tq, at):
    L, x, w = tq.lib(), tq._Mat(FAKE, 1, 0, 1, 40, 128, 128, 0), records(tq, tq.INT4_G64_ASYM)
    assert refused(tq, L.tq_head_loss(R(w), R(x), FAKE, at, FAKE, FAKE, BIG, None))
    assert refused(tq, L.tq_head_loss(R(w), R(x), FAKE, FAKE, at, FAKE, BIG, None))
    assert refused(tq, L.tq_head_loss_backward(R(w), R(x), FAKE, at, FAKE, FAKE, 128, FAKE, BIG, None))
    assert refused(tq, L.tq_head_loss_backward(R(w), R(x), FAKE, FAKE, at, FAKE, 128, FAKE, BIG, None))
