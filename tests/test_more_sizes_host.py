"""Integers beyond 32 bits are refused by the grouped router's binding, not cut to their low half (no GPU)."""
import pytest
import torch

from moe_task_scheduling_gb300 import etmoe as E
from tests.test_sizes_host import WS, Told

F32, I32 = torch.float32, torch.int32


def _forward(**over):
    a = dict(score=E.ET_SCORE_SIGMOID, n_groups=4, k_groups=2, group_best=2)
    a.update(over)
    E.et_router_groups(Told(4, 8, dtype=F32), Told(4, 2, dtype=I32), Told(4, 2, dtype=F32), workspace=WS, **a)


def _backward(score):
    E.et_router_groups_bwd(Told(4, 8, dtype=F32), Told(4, 2, dtype=I32), Told(4, 2, dtype=F32), Told(8, dtype=I32), Told(1, dtype=I32),
                           Told(4, 8, dtype=F32), score=score, workspace=WS)


@pytest.mark.parametrize("wide", [1 << 32, -(1 << 32)])  # added to a value that the calls accept
def test_wide_choices_are_refused(wide):
    for over in (dict(score=wide), dict(score=wide + 1), dict(n_groups=wide + 4), dict(k_groups=wide + 2), dict(group_best=wide + 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            _forward(**over)
    for score in (wide, wide + 1):
        with pytest.raises(ValueError, match="2\\^31"):
            _backward(score)
