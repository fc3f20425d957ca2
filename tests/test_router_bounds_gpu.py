"""et_router_topk's stated error bounds where they are tight: the logarithm near zero, weights far
below the largest."""
import pytest
import torch

from tests import ref_ops as ref
from tests.test_router_gpu import _backward, _forward

pytestmark = pytest.mark.gpu
U = ref.F32_HALF


def test_logarithm_near_zero(cuda_lib):
    """Rows (0, -d): log(sum exp) runs from log 2 down to nothing, seen row by row in the z loss' gradient
    2 / n * lse * p."""
    T = 4096
    d = torch.linspace(0, 18, T)
    logits = torch.stack((torch.zeros(T), -d), 1)
    o, ws, L, m = _forward(cuda_lib, logits, 1)
    dl = torch.tensor([0.0, T / 2])
    got = _backward(cuda_lib, o, ws, L, m, dl, None)
    p = torch.softmax(logits.double(), -1)
    lse = torch.logsumexp(logits.double(), -1, keepdim=True)
    # log: 2^-21.4 at most between 1/2 and 2; its argument s: half a step and what exp is off, (4 + 2.4 d) e^-d;
    # p: exp, s and the quotient's 2 ulp; two products
    e = (4 + 2.4 * d.double()[:, None]) * torch.exp(-d.double()[:, None]) * U
    lse_err = 2 ** -21.4 + (1.0 * U + e) + 2 * U * lse
    p_rel = (4 + 2.4 * d.double()[:, None] * torch.tensor([0.0, 1.0]) + 2 + 4 + 4) * U + e
    ref.check(got, lse * p, p * lse_err + lse * p * p_rel + 1e-38, "d_logits")


@pytest.mark.parametrize("En", [2, 40, 100])
def test_weights_far_below_the_largest(cuda_lib, En):
    """Rows (0, -d, -inf ...): the second weight runs from 1/2 down to e^-80.  L - L0 is exact here; exp is off by 1 ulp,
    the sum by half a step and the exp in it, the quotient by half a step."""
    T = 8192
    d = torch.linspace(0, 80, T)
    logits = torch.full((T, En), -float("inf"))
    logits[:, 0], logits[:, 1] = 0, -d
    o, _, _, _ = _forward(cuda_lib, logits, 2)
    want = torch.softmax(logits[:, :2].double(), -1)
    exp = torch.tensor([0.0, 2.0]) + 2 * torch.exp(-d.double()[:, None])
    ref.check(o["w"], want, (exp + 2) * U * want, "w")
