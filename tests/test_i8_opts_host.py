"""et_i8_gemm_opts without a GPU: the refusals of et_i8_gemm, with and without options."""
import ctypes

import pytest

from moe_task_scheduling_gb300 import etmoe as E

GEMM = dict(x=16, sx=16, w=16, sw=16, Y=16, M=2, dM=None, Mm=4, N=64, K=64, ws=256, wsb=1 << 40)


@pytest.mark.parametrize("over,code", [(dict(x=None), E.ET_ERR_INVALID), (dict(w=24), E.ET_ERR_INVALID), (dict(Y=17), E.ET_ERR_INVALID),
                                       (dict(M=5), E.ET_ERR_INVALID), (dict(K=24), E.ET_ERR_UNSUPPORTED),
                                       (dict(Mm=0), E.ET_ERR_UNSUPPORTED), (dict(ws=None), E.ET_ERR_WORKSPACE),
                                       (dict(wsb=100), E.ET_ERR_WORKSPACE), (dict(M=0), E.ET_OK)])
def test_the_same_refusals(over, code):
    import __graft_entry__
    __graft_entry__.build()
    a = list(dict(GEMM, **over).values())
    lib = E.load()
    assert lib.et_i8_gemm(*a, None) == code
    assert lib.et_i8_gemm_opts(*a, None, None) == code
    assert lib.et_i8_gemm_opts(*a, ctypes.byref(E.et_opts(1000, 0, 1, 0, None)), None) == code
