"""The bound that the 4-bit experts are checked with shows what a faulty kernel would lose (no GPU)."""
import pytest
import torch

from tests import ref_w4


@pytest.mark.parametrize("T,H,F,En,k,group", ref_w4.SIZES)
def test_a_lost_part_breaks_the_check(T, H, F, En, k, group):
    a = ref_w4.inputs(T, H, F, En, k, group, T + H)
    want, bound = ref_w4.experts(*a)
    tol = ref_w4.tolerance(want, bound)
    assert float(bound.max()) < 0.05 * float(want.square().mean().sqrt())
    rounded = want.to(torch.bfloat16).double()
    assert ((rounded - want).abs() <= tol).all()
    for drop in ("row", "up", "down"):
        got = ref_w4.experts(*a, drop=drop)[0].to(torch.bfloat16).double()
        assert int(((got - want).abs() > tol).sum()) > H // 4, drop


def test_gate_and_up_are_exact():
    """Every partial sum of an expert's gate and up products is a value of fp32."""
    from tests.ref_ops import w4_values
    x, idx, w, gate, up, down = ref_w4.inputs(2, 4128, 96, 2, 2, 32, 1)
    for q, s in (gate, up):
        terms = x[0].double() * w4_values(q[0], s[0])
        assert torch.equal(terms.cumsum(-1).float().double(), terms.cumsum(-1))
        unit = float(s[0].double().min())
        assert float(terms.abs().sum(-1).max()) / unit < 2 ** 24
