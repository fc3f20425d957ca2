"""et_router_groups where distinct logits have scores that are equal in 64 bits: the lower index, whatever path a row takes."""
import math

import pytest
import torch

from tests import ref_more as ref

pytestmark = pytest.mark.gpu

# 0.5 as sigmoid scores, and 1 as e^x, in 64 bits: half a step is 2^-54 there
TINY = torch.tensor([0.0, 1e-20, -1e-20, 1e-17, -1e-17, 1e-25, -0.0, 1e-40, -1e-40, 3e-30])


def _idx(E, L, k, G, kg, best, sigmoid, bias):
    T, En = L.shape
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ws = E.alloc_workspace(E.et_router_groups_workspace_bytes(T, En, k))
    E.et_router_groups(L.cuda(), idx, w, score=E.ET_SCORE_SIGMOID if sigmoid else E.ET_SCORE_SOFTMAX, n_groups=G, k_groups=kg,
                       group_best=best, bias=None if bias is None else bias.cuda(), workspace=ws)
    assert E.et_status(ws) == (0, 0)
    return idx.cpu().long()


def _rows(T, En, g):
    """Logits around 0 that tie among ones that do not, a different number of either in each row."""
    tiny = TINY[torch.randint(0, len(TINY), (T, En), generator=g)]
    far = torch.randn(T, En, generator=g)
    far = torch.where(far.abs() < 1e-3, torch.ones(()), far)
    L = torch.where(torch.rand(T, En, generator=g) < torch.rand(T, 1, generator=g), tiny, far)
    i = torch.arange(T) % 8
    L[i == 1] = -L[i == 1].abs()                                    # the ties are the best,
    L[i == 2] = tiny[i == 2]                                        # or all there is
    L[i == 3, En // 3] = 20.0                                       # with logits far above:
    L[i == 4] = torch.where(torch.rand(int((i == 4).sum()), En, generator=g) < 0.1, 18 + far[i == 4].abs(), tiny[i == 4])
    L[i == 5] = torch.where(torch.rand(int((i == 5).sum()), En, generator=g) < 0.1, 45 + far[i == 5], L[i == 5])
    L[i == 6, ::3] = -math.inf
    return L


@pytest.mark.parametrize("En,k,G,kg", [(3, 1, 1, 1), (8, 2, 1, 1), (30, 4, 5, 3), (32, 8, 8, 4), (64, 6, 1, 1), (128, 8, 8, 4), (160, 8, 5, 2),
                                       (256, 8, 1, 1), (256, 8, 8, 4)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [None, "zero"])
def test_scores_that_meet(cuda_lib, En, k, G, kg, sigmoid, bias):
    g = torch.Generator().manual_seed(En + k)
    L = _rows(1100, En, g)
    b = None if bias is None else torch.zeros(En)
    for best in (1, 2):
        want = ref.router_groups(L[:400], k, G, kg, best, sigmoid=sigmoid, bias=b)["idx"]
        many = _idx(cuda_lib, L, k, G, kg, best, sigmoid, b)  # from 1024 rows on four may share a warp
        few = torch.cat([_idx(cuda_lib, L[t:t + 300], k, G, kg, best, sigmoid, b) for t in range(0, 1100, 300)])
        assert torch.equal(many, few)
        assert torch.equal(many[:400], want)


@pytest.mark.parametrize("T", [5, 1030])
def test_differences_lost_to_the_largest_logit(cuda_lib, T):
    """e^(x - max) of logits that differ by less than their distance from the largest one's last bit."""
    L = torch.full((T, 32), -math.inf)
    L[:, 0] = 300.0
    L[:, 1:9] = torch.tensor([0.0, 1e-16, -1e-16, 2e-15, 0.0, -2e-15, 1e-14, 1e-20])
    # 300 - x in 64 bits has steps of 2^-44 = 5.7e-14: one value for all eight
    got = _idx(cuda_lib, L, 6, 1, 1, 1, False, None)
    assert torch.equal(got, torch.arange(6).expand(T, 6))
