"""Refusals of the operators' entry points on the host, beside
test_ops_boundary.py: gradients of an fp32 result, sizes past 64 bits."""
import pytest

import dense_tiled_gemm_tgemm_amd as tg

INV = tg.TGEMM_ERR_INVALID
# fake, well-separated, aligned device addresses (never dereferenced)
P = [(i + 1) << 42 for i in range(12)]


def act_grad(**kw):
    a = dict(M=64, N=96, type="f16", dY=P[0], lddy=96, act="gelu", pre=P[1], ldpre=96, dP=P[2], lddp=96, scale=P[5],
             dbias_type="f32", dbias=P[3], workspace=P[4], workspace_bytes=1 << 30)
    a.update(kw)
    return tg.tgemm_act_grad_f32(**a)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(type="f32"), dict(act=7), dict(dbias_type="bf16"), dict(lddy=95), dict(ldpre=95), dict(lddp=95),
    dict(pre=None), dict(dP=None), dict(scale=None), dict(act="none"), dict(dP=P[0]), dict(dP=P[1] + 2), dict(dbias=P[0]),
    dict(dY=P[0] + 2), dict(dP=P[2] + 1), dict(scale=P[5] + 2), dict(scale=P[0] + 4), dict(scale=P[2] + 4), dict(dbias=P[2]),
    dict(workspace=None), dict(workspace_bytes=16), dict(workspace_bytes=4 * 96 * 4), dict(workspace=P[4] + 8),
    dict(workspace=P[0]), dict(workspace=P[2])])
def test_act_grad_f32_refuses(kw):
    assert act_grad(**kw) == INV


def test_act_grad_f32_accepts_empty_problems_without_a_device():
    assert act_grad(N=0) == tg.TGEMM_OK
    assert act_grad(M=0, dbias=None) == tg.TGEMM_OK
    assert act_grad(dP=None, scale=None, dbias=None) == tg.TGEMM_OK
    assert tg.tgemm_act_grad_f32_workspace(-1, 8) == INV
    assert tg.tgemm_act_grad_f32_workspace(0, 8) >= 0


def linear_grad(**kw):
    a = dict(M=64, N=96, K=128, type="bf16", X=P[0], ldx=128, W=P[1], ldw=128, w_layout="NxK", act="gelu", pre=P[2],
             ldpre=96, dY=P[3], lddy=96, dX=P[4], lddx=128, dW=P[5], lddw=128, dbias_type="bf16", dbias=P[6],
             workspace=P[7], workspace_bytes=1 << 40)
    a.update(kw)
    return tg.tgemm_linear_grad_f32(**a)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(type="f32"), dict(w_layout=3), dict(act=-2), dict(dbias_type="f16"), dict(ldx=127), dict(ldw=127),
    dict(lddy=95), dict(ldpre=95), dict(lddx=127), dict(lddw=127), dict(pre=None), dict(act="none"), dict(X=None),
    dict(dY=None), dict(dY=P[3] + 2), dict(dX=P[0]), dict(dW=P[1]), dict(dX=P[5]), dict(dbias=P[4]), dict(dW=P[3] + 2)])
def test_linear_grad_f32_refuses(kw):
    assert linear_grad(**kw) == INV


def test_workspaces_past_63_bits_are_refused():
    """Sizes that the header allows and no memory holds: refused, not wrapped."""
    big, UNS = 2 ** 31 - 1, tg.TGEMM_ERR_UNSUPPORTED
    assert tg.tgemm_linear_workspace(big, big, 4, "bf16", 4, 4, "NxK", "bf16", big) == UNS
    assert tg.tgemm_tn_workspace(big, big, 4, "bf16", big, big, "bf16", big) == UNS
    for query in (tg.tgemm_linear_grad_workspace, tg.tgemm_linear_grad_f32_workspace):
        for act in ("none", "silu"):
            assert query(big, big, 4, "bf16", 4, 4, "NxK", act, big, 4, 4) == UNS
            assert query(big, 4, big, "bf16", big, big, "NxK", act, 4, big, big) == UNS
            assert query(4, big, big, "bf16", big, big, "NxK", act, big, big, big) == UNS
    assert tg.tgemm_linear_workspace(big, 0, 4, "bf16", 4, 4, "NxK", "bf16", 1) == 0
