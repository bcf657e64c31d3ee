"""A step with PKV_STEP_OVERLAP may read lengths that any kernel but the one just
before it wrote.  Acceptance writes new lengths; a scored call, a tree call or an
eviction of other sequences stands between it and the step.  The lengths change at
every round, and each round has to give, bit for bit, what the same calls give with a
wait after each (single-token decode is repeatable, and so are weights)."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, MBS = 200, 8, 4, 64, 8


class State:
    def __init__(self):
        g = torch.Generator().manual_seed(3)
        NB = B * MBS

        def draw(*shape):
            return torch.randn(*shape, generator=g).half().cuda()

        self.kc, self.vc = draw(NB, HKV, 16, D), draw(NB, HKV, 16, D)
        self.q, self.k, self.v = draw(B, HQ, D), draw(B, HKV, D), draw(B, HKV, D)
        self.tq = draw(8 * B, HQ, D)
        self.tables = torch.randperm(NB, generator=g).view(B, MBS).int().cuda()
        self.desc = pkv.make_desc(NB, 16, HKV, HQ, D, pkv.PKV_F16)
        i = dict(dtype=torch.int32, device="cuda")
        # two sets of lengths in turn: 8 nodes behind pasts of 8 to 112 tokens
        self.ctx = [(8 + torch.randint(8, 113, (B,), generator=g)).int().cuda() for _ in range(2)]
        self.starts = (8 * torch.arange(B + 1)).int().cuda()
        self.path = torch.arange(7, -1, -1).int().repeat(B, 1).cuda()
        self.accepted = [torch.randint(1, 9, (B,), generator=g).int().cuda() for _ in range(2)]
        self.mask = (torch.arange(8 * B) % 8).apply_(lambda j: (2 << j) - 1).cuda()
        self.weights = torch.zeros(NB, HKV, 16, device="cuda")
        self.positions = torch.zeros(NB, HKV, 16, **i)
        self.new, self.evicted, self.zero = (torch.zeros(B, **i) for _ in range(3))
        self.outs = [torch.zeros(B, HQ, D, device="cuda") for _ in range(2)]
        self.tree_out = torch.zeros(8 * B, HQ, D, device="cuda")
        self.sws = torch.zeros(pkv.pkv_scored_workspace_bytes(self.desc, B, MBS),
                               dtype=torch.uint8, device="cuda")
        self.dws = torch.zeros(pkv.pkv_decode_workspace_bytes(self.desc, B, MBS),
                               dtype=torch.uint8, device="cuda")
        self.tws = torch.zeros(pkv.pkv_tree_workspace_bytes(self.desc, B, 8, MBS),
                               dtype=torch.uint8, device="cuda")

    def round(self, turn, between, overlap, wait):
        pkv.pkv_kv_accept_path(self.desc, self.kc, self.vc, self.tables, self.ctx[turn],
                               self.starts, self.path, self.accepted[turn], self.new)
        wait()
        if between == "scored":
            pkv.pkv_paged_decode_attention_scored(self.desc, self.q, self.kc, self.vc, self.tables,
                                                  self.ctx[0], self.weights, 0.125, self.outs[0],
                                                  self.sws, decay=0.5)
        elif between == "tree":
            pkv.pkv_paged_tree_attention(self.desc, self.tq, self.kc, self.vc, self.tables,
                                         self.ctx[0], self.starts, 8, self.mask, 0.125,
                                         self.tree_out, self.tws)
        else:
            pkv.pkv_kv_evict(self.desc, self.kc, self.vc, self.weights, self.positions, self.tables,
                             self.ctx[0], self.zero, self.ctx[0], 100, 4, 8, self.evicted)
        wait()
        pkv.pkv_decode_step_fused(self.desc, self.q, self.kc, self.vc, self.k, self.v, self.tables,
                                  self.new, 0.125, self.outs[1], self.dws, overlap=overlap)
        wait()

    def results(self):
        return [self.kc, self.vc, self.weights, self.positions, self.new, self.evicted,
                self.tree_out, *self.outs]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("between", ["scored", "tree", "evict"])
def test_lengths_of_an_earlier_kernel(between, graph):
    ref, got = State(), State()
    run = [lambda t=t: got.round(t, between, True, lambda: None) for t in range(2)]
    if graph:
        graphs = []
        for f in run:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            graphs.append(g)
        run = [g.replay for g in graphs]
    torch.cuda.synchronize()
    for step in range(12):
        ref.round(step % 2, between, False, torch.cuda.synchronize)
        run[step % 2]()
        torch.cuda.synchronize()
        for x, y in zip(got.results(), ref.results()):
            assert torch.equal(x, y), step
    for step in range(40):  # rounds in a row, without a wait between them
        run[step % 2]()
        ref.round(step % 2, between, False, lambda: None)
    torch.cuda.synchronize()
    for x, y in zip(got.results(), ref.results()):
        assert torch.equal(x, y)
