"""Router, 4-bit conversion and experts many times back to back, nothing waited for on the host: every step's experts
see that step's indices, weights, count and rows, in one set of buffers that each step writes anew."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Steps:
    def __init__(self, E, T, H, F, En, k, group, n, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.n = E, n
        self.logits = torch.randn(n, T, En, generator=g, device="cuda")
        self.rows = torch.randn(n, T, H, generator=g, device="cuda").to(BF)
        self.counts = torch.randint(1, T + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        self.w = [[(torch.randn(En, N, K, generator=g, device="cuda") / K ** 0.5).to(BF) for N, K in ((F, H), (F, H), (H, F))] for _ in range(2)]
        self.q = [t for N, K in ((F, H), (F, H), (H, F)) for t in (torch.zeros(En, N, K // 2, dtype=torch.uint8, device="cuda"),
                                                                   torch.zeros(En, K // group, N, dtype=BF, device="cuda"))]
        self.x, self.L = torch.zeros(T, H, dtype=BF, device="cuda"), torch.zeros(T, En, device="cuda")
        self.idx, self.gw = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        self.dT = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.wsr = E.alloc_workspace(E.et_router_topk_workspace_bytes(T, En, k))
        self.wse = E.alloc_workspace(E.et_w4_experts_workspace_bytes(T, H, F, En, k, group))
        self.out = torch.full((n, T, H), 7.0, dtype=BF, device="cuda")

    def step(self, i, weights):
        E = self.E
        self.x.copy_(self.rows[i])
        self.L.copy_(self.logits[i])
        if weights:
            for j, w in enumerate(self.w[i % 2]):
                E.et_w4_quantize(w, self.q[2 * j], self.q[2 * j + 1])
        self.dT.copy_(self.counts[i:i + 1])
        E.et_router_topk(self.L, self.idx, self.gw, d_T=self.dT, workspace=self.wsr)
        E.et_w4_experts(self.x, self.idx, self.gw, *self.q, self.out[i], d_T=self.dT, workspace=self.wse)


@pytest.mark.parametrize("T,H,F,En,k,group", [(1, 512, 256, 64, 8, 128), (4, 256, 512, 8, 2, 64), (12, 512, 256, 64, 8, 32),
                                              (40, 448, 320, 250, 8, 64), (24, 1536, 256, 16, 8, 128)])
@pytest.mark.parametrize("weights", [False, True])
def test_every_step_sees_its_own_inputs(cuda_lib, T, H, F, En, k, group, weights):
    s = Steps(cuda_lib, T, H, F, En, k, group, 60, T + H)
    for j in range(3):
        cuda_lib.et_w4_quantize(s.w[0][j], s.q[2 * j], s.q[2 * j + 1])
    for i in range(s.n):  # one at a time, waited for
        s.step(i, weights)
        torch.cuda.synchronize()
    want = s.out.clone()
    for r in range(4):
        s.out.fill_(7)
        for i in range(s.n):
            s.step(i, weights)
        assert torch.equal(s.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(s.n):
            s.step(i, weights)
    for r in range(4):
        s.out.fill_(7)
        g.replay()
        assert torch.equal(s.out, want)
    assert cuda_lib.et_status(s.wse) == (0, 0) and cuda_lib.et_status(s.wsr) == (0, 0)
    assert (s.wse[8:256] == 0).all()  # every counter is back at zero
