"""et_router_topk's sums over many tokens against the 64-bit definitions."""
import pytest
import torch

from tests import ref_ops as ref
from tests.test_router_gpu import _forward, _gen

pytestmark = pytest.mark.gpu
U = ref.F32_HALF


@pytest.mark.parametrize("T,En,k", [(155648, 8, 2), (155649, 8, 2), (200001, 8, 2), (700003, 8, 2), (330007, 72, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_second_level_of_sums(cuda_lib, T, En, k, masked):
    """A warp adds up 32 rows, then those sums: from 152 CTAs x 32 warps x 32 rows = 155648 tokens on the second
    level is used, with one flush, several, and a rest behind the last."""
    g = _gen(T)
    logits = torch.randn(T, En, generator=g) * 2
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if masked else None
    o, ws, _, _ = _forward(cuda_lib, logits, k, mask)
    r = ref.router(logits, k, mask)
    assert torch.equal(o["idx"].cpu(), r["idx"].to(torch.int32))
    assert torch.equal(o["counts"].cpu(), r["counts"].to(torch.int32)) and int(o["n"]) == r["n"]
    # of a probability: exp (2 + 1.2 |L - L0| ulp) and its argument, the sum of E, two quotients; of a sum: 32
    # additions, then one for each 32 rows of a warp, 32 warps, 152 CTAs in 19s and eights, a quotient; each at
    # most half a step
    spread = float(logits.max() - logits.min())
    row = (12 + 4 * spread + En) * U
    depth = (32 + T / (152 * 32 * 32) + 32 + 19 + 8 + 4) * U
    ref.check(o["mean_prob"], r["mean_prob"], (row + depth) * r["mean_prob"], "mean_prob")
    # log(sum): 2^-21.4 (up to s = 2) or 3 ulp, L0 added; squared
    lse_err = 2 ** -21.4 + (8 * r["lse"].abs() + 2 * logits.double().abs().max(-1).values + En + 4) * U
    n = max(r["n"], 1)
    z_err = 2 * (r["lse"].abs() * torch.where(r["live"], lse_err, 0.0)).sum() / n + (depth + 4 * U) * r["losses"][1]
    ref.check(o["losses"], r["losses"], torch.stack(((row + depth + (En + 8) * U) * r["losses"][0], z_err)), "losses")
    o2, _, _, _ = _forward(cuda_lib, logits, k, mask, ws=ws)
    assert all(torch.equal(o[name], o2[name]) for name in o)
