"""Sizes and counts beyond 32 bits are refused by the binding, not cut to their low half (no GPU: tensors that only
tell their shape)."""
import pytest
import torch

from moe_task_scheduling_gb300 import etmoe as E

BIG = (1 << 32) + 8  # its low half is a size that the calls accept


class Told:
    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def numel(self):
        return 1 << 40

    def dim(self):
        return len(self.shape)


F32, I32, U8 = torch.float32, torch.int32, torch.uint8
WS = Told(1 << 40, dtype=U8)


def _router(T=4, En=8, rows=None):
    E.et_router_topk(Told(T, En, dtype=F32), Told(T, 2, dtype=I32), Told(T, 2, dtype=F32), T=rows, workspace=WS)


def _router_bwd(T=4, En=8, rows=None):
    E.et_router_topk_bwd(Told(T, En, dtype=F32), Told(T, 2, dtype=I32), Told(T, 2, dtype=F32), Told(En, dtype=I32),
                         Told(1, dtype=I32), Told(T, En, dtype=F32), T=rows, workspace=WS)


def _norm(T=4, H=8, rows=None):
    E.et_block_norm(Told(T, H), None, Told(T, H), None, eps=1e-5, T=rows, workspace=WS)


def _norm_bwd(T=4, H=8, rows=None):
    E.et_block_norm_bwd(Told(T, H), None, Told(T, H), None, Told(T, H), None, eps=1e-5, T=rows, workspace=WS)


def _gemv(M=4, N=8, K=64, rows=None):
    E.et_w4_gemv(Told(M, K), Told(N, K // 2, dtype=U8), Told(K // 32, N), Told(M, N), M=rows, workspace=WS)


def _experts(T=4, H=64, F=64, rows=None):
    w = [Told(8, n, k // 2, dtype=U8) if i == 0 else Told(8, k // 32, n) for n, k in ((F, H), (F, H), (H, F)) for i in (0, 1)]
    E.et_w4_experts(Told(T, H), Told(T, 2, dtype=I32), Told(T, 2, dtype=F32), *w, Told(T, H), T=rows, workspace=WS)


def _quantize(En=1, N=8, K=64):
    E.et_w4_quantize(Told(En, N, K), Told(En, N, K // 2, dtype=U8), Told(En, K // 32, N))


def _dequantize(En=1, N=8, K=64):
    E.et_w4_dequantize(Told(En, N, K // 2, dtype=U8), Told(En, K // 32, N), Told(En, N, K))


WIDE = BIG + 56  # low half 64: a multiple of 32
CASES = [(_router, dict(T=BIG)), (_router, dict(En=BIG)), (_router, dict(rows=BIG)), (_router, dict(rows=4 - (1 << 32))),
         (_router_bwd, dict(T=BIG)), (_router_bwd, dict(En=BIG)), (_router_bwd, dict(rows=(1 << 32) + 1)),
         (_norm, dict(T=BIG)), (_norm, dict(H=BIG)), (_norm, dict(rows=1 << 32)),
         (_norm_bwd, dict(T=BIG)), (_norm_bwd, dict(H=BIG)), (_norm_bwd, dict(rows=1 << 32)),
         (_gemv, dict(M=BIG)), (_gemv, dict(N=BIG)), (_gemv, dict(K=WIDE)), (_gemv, dict(rows=1 << 32)),
         (_experts, dict(T=BIG)), (_experts, dict(H=WIDE)), (_experts, dict(F=WIDE)), (_experts, dict(rows=1 << 32)),
         (_quantize, dict(En=BIG)), (_quantize, dict(N=BIG)), (_quantize, dict(K=WIDE)),
         (_dequantize, dict(N=BIG)), (_dequantize, dict(K=WIDE))]


@pytest.mark.parametrize("call,over", CASES)
def test_sizes_beyond_32_bits_are_refused(call, over, monkeypatch):
    def reached(*a):
        raise AssertionError("the call went on to the library")
    monkeypatch.setattr(E, "_call", reached)
    with pytest.raises(AssertionError, match="went on"):  # the same call of ordinary sizes does
        call()
    with pytest.raises(ValueError):
        call(**over)


def test_workspace_of_sizes_beyond_32_bits():
    import __graft_entry__
    __graft_entry__.build()
    assert E.et_router_topk_workspace_bytes(BIG, 8, 2) == 0 and E.et_block_norm_workspace_bytes(4, BIG) == 0
    assert E.et_w4_gemv_workspace_bytes(4, BIG, 64, 32) == 0 and E.et_w4_gemv_workspace_bytes(4, 8, 64, 32 - (1 << 32)) == 0
    assert E.et_w4_experts_workspace_bytes(4, 64, WIDE, 8, 2, 32) == 0
