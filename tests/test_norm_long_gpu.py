"""et_block_norm_bwd over so many rows that the parameter gradients are summed by several launches."""
import pytest
import torch

from tests import ref_ops as ref

pytestmark = pytest.mark.gpu
U = ref.F32_HALF
BF = torch.bfloat16
EPS = 1e-5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bwd(E, x, y, dz, dh, par, wanted=True, T=None, d_T=None):
    Tm, H = x.shape
    o = dict(dx=torch.full_like(x, 7.0), dy=torch.full_like(x, 7.0))
    for n in ("d_gamma_post", "d_gamma_pre", "d_gate"):
        o[n] = torch.full((H,), 7.0, device="cuda") if wanted else None
    ws = E.alloc_workspace(E.et_block_norm_workspace_bytes(Tm, H))
    E.et_block_norm_bwd(x, y, dz, dh, scale=0.5, eps=EPS, T=T, d_T=d_T, workspace=ws, **par, **o)
    assert E.et_status(ws) == (0, 0)
    return o


def _par(H, seed):
    g = _gen(seed)
    return {n: (m + 0.1 * torch.randn(H, generator=g)).to(BF).cuda() for n, m in (("gamma_post", 1.0), ("gamma_pre", 1.0), ("gate", 0.5))}


# rows of a launch: 256 for each of 304 CTAs (152 with more than 256 threads) and row groups
@pytest.mark.parametrize("T,H,unstaged", [(500000, 2056, False), (500000, 2056, True), (300000, 2061, False), (4000000, 256, False),
                                          (3000000, 130, False), (4000000, 256, True), (1500000, 520, False), (200000, 4104, False)])
def test_equal_rows(cuda_lib, T, H, unstaged):
    """All rows alike: the sums are T times one row's, and every addition of a chain rounds the same way."""
    g = _gen(H)
    rows = [torch.randn(1, H, generator=g).to(BF).cuda() for _ in range(4)]
    if unstaged:
        rows[2] = None
    par = _par(H, H)
    one = _bwd(cuda_lib, *rows, par)
    many = _bwd(cuda_lib, *[None if r is None else r.expand(T, H).contiguous() for r in rows], par)
    # 256 rows of a thread, up to 8 row groups, 304 CTAs in tens and fives, T / (256 * 152) launches; and one row's own
    depth = 256 + 8 + 10 + 5 + T / (256 * 152) + 2
    for n in ("d_gamma_post", "d_gamma_pre", "d_gate"):
        want = T * one[n].double()
        ref.check(many[n], want, depth * U * want.abs() + 1e-30, n)
    for n in ("dx", "dy"):
        assert (many[n] == one[n]).all()


@pytest.mark.parametrize("T,H", [(170000, 2056), (78000, 4104), (700000, 264)])
def test_several_launches_are_one(cuda_lib, T, H):
    """Two or three launches: dx and dy are the bits of a call without parameter gradients, which is one launch; the
    gradients are the sum of those over the rows' halves; a device count ends within any of them."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x, y, dz, dh = (torch.randn(T, H, generator=g, device="cuda").to(BF) for _ in range(4))
    par = _par(H, T)
    whole, bare = _bwd(cuda_lib, x, y, dz, dh, par), _bwd(cuda_lib, x, y, dz, dh, par, wanted=False)
    assert torch.equal(whole["dx"], bare["dx"]) and torch.equal(whole["dy"], bare["dy"])
    again = _bwd(cuda_lib, x, y, dz, dh, par)
    cut = T // 3
    parts = [_bwd(cuda_lib, *(v[a:b] for v in (x, y, dz, dh)), par) for a, b in ((0, cut), (cut, T))]
    d_T = torch.full((1,), cut, dtype=torch.int32, device="cuda")
    short = _bwd(cuda_lib, x, y, dz, dh, par, d_T=d_T)
    host = _bwd(cuda_lib, x, y, dz, dh, par, T=cut)
    for n in ("d_gamma_post", "d_gamma_pre", "d_gate"):
        assert torch.equal(whole[n], again[n])
        # random signs: the magnitudes added up are T times one of order one; two sums of at most 300 additions each
        ref.check(whole[n], parts[0][n].double() + parts[1][n].double(), 2 * 300 * U * 8 * T, n)
        ref.check(short[n], parts[0][n].double(), 2 * 300 * U * 8 * T, n)
        ref.check(host[n], parts[0][n].double(), 2 * 300 * U * 8 * T, n)
    for o in (short, host):
        assert torch.equal(o["dx"][:cut], whole["dx"][:cut]) and (o["dx"][cut:] == 7).all() and (o["dy"][cut:] == 7).all()
    d_T.fill_(0)
    none = _bwd(cuda_lib, x, y, dz, dh, par, d_T=d_T)
    assert all((none[n] == 0).all() for n in ("d_gamma_post", "d_gamma_pre", "d_gate")) and (none["dx"] == 7).all()
