"""Workspaces whose status word is not on a boundary are refused (the kernels would fault when they write it)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def M():
    import moe_expert_ffn_sqrt_gb300 as M
    if not os.path.exists(M.LIB_PATH):
        from moe_expert_ffn_sqrt_gb300 import build
        build.build()
    M.lib()
    return M


P = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
BIG = 1 << 40
ODD = ctypes.c_void_p(0x10002)


def calls(M):
    """name -> (call(ws, one of its int32 or float arrays), whether it has a workspace, the arrays' names)"""
    L = M.lib()
    r = lambda ld=64: M._Rows(0x10000, ld)   # noqa: E731
    r8 = M._Rows8(0x10000, 0x20000, 64, 1)
    none, none8 = M._Rows(None, 0), M._Rows8(None, None, 0, 0)

    def dispatch(ws=P, ids=P, sorted_ids=P, experts=P, inv=P, m_sum=P, counts=P):
        return L.moe_dispatch(0, ids, r(), 4, 64, 8, 2, 16, r(), sorted_ids, experts, inv, m_sum, counts, ws, BIG, None)

    def combine(ws=P, inv=P, w=P):
        return L.moe_combine(0, r(), inv, w, none, 4, 64, 2, 64, r(), ws, BIG, None)

    def combine_backward(ws=P, inv=P, w=P, dw=P):
        return L.moe_combine_backward(0, r(), r(), inv, w, 4, 64, 2, 64, r(), dw, ws, BIG, None)

    def dispatch_backward(ws=P, inv=P):
        return L.moe_dispatch_backward(0, r(), inv, none, 4, 64, 2, 64, r(), ws, BIG, None)

    def route_backward(ws=P, ids=P, w=P, dw=P):
        return L.moe_route_backward(P, ids, w, dw, 4, 64, 2, 0, 1, 0, P, ws, BIG, None)

    def select(bias=P, ids=P, w=P):
        return L.moe_select(2, r(), bias, 4, 64, 6, M._SelectRule(2, 8, 4, 2, 1, 1.0), ids, w, None)

    def select_backward(ws=P, ids=P, w=P, dw=P):
        return L.moe_select_backward(2, r(), ids, w, dw, 4, 64, 6, 2, 1, 1.0, 2, r(), ws, BIG, None)

    def pack(ws=P, counts=P):
        return L.moe_pack_rows8(0, r(), counts, 4, 64, 2, 4, r8, ws, BIG, None)

    def unpack(ws=P, counts=P, ids=P):
        return L.moe_unpack_rows8(0, r8, ids, 1, 4, counts, 4, 64, 2, 4, r(), ws, BIG, None)

    def linear(ws=P, counts=P):
        return L.moe_linear(0, r(), P, None, none, 0, counts, 4, 64, 64, 2, 4, r(), none, ws, BIG, None)

    def linear_backward(ws=P, counts=P):
        return L.moe_linear_backward(0, r(), r(), P, none, 0, counts, 4, 64, 64, 2, 4, none, r(), P, None, ws, BIG, None)

    def linear_backward8(ws=P, counts=P, ids=P):
        return L.moe_linear_backward8(0, r(), none, r8, ids, 1, 4, P, none, none8, 0, counts, 4, 64, 64, 2, 4, none, r(), P, None, ws,
                                      BIG, None)

    def norm_backward(ws=P):
        return L.moe_rms_norm_backward(0, r(), r(), P, 1e-6, none, 4, 64, r(), P, ws, BIG, None)

    return [dispatch, combine, combine_backward, dispatch_backward, route_backward, select, select_backward, pack, unpack, linear,
            linear_backward, linear_backward8, norm_backward]


@pytest.mark.parametrize("i", range(13))
def test_arrays_off_their_elements_boundary_are_refused(M, i):
    f = calls(M)[i]
    names = f.__code__.co_varnames[:f.__code__.co_argcount]
    assert names
    for n in names:
        want = M.ERR_WORKSPACE if n == "ws" else M.ERR_INVALID_ARG
        assert f(**{n: ODD}) == want, (f.__name__, n)
