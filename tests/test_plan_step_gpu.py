"""A decode step on the slot map that a batch plan has just written: the step's launch may start while the
plan's kernel still runs, and reads nothing of it before that kernel's writes are visible."""
import numpy as np
import pytest
import torch

import quantized_linear_attention_damp_b200 as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n,H", [(4, 2), (96, 16)])
def test_steps_on_slots_of_plans_just_built(n, H, captured):
    """24 rounds of plan, then step on its store_slot, with no synchronisation between them, each with other
    slots, other requests without a token and other gates, against steps on slots from the host."""
    d, n_slots, rounds = 128, n + 3, 24
    g = np.random.default_rng(n)
    rows = np.stack([np.sort(g.permutation(d)[:27]) for _ in range(H)])
    pools = [D.DampPool("mixed", n_slots, H, d, rows) for _ in range(2)]
    cpu = torch.Generator().manual_seed(n)
    S0 = torch.randn(n_slots, H, d, d, generator=cpu).cuda() * 0.2
    for p in pools:
        p.slots().zero_()
        p.pack(torch.arange(n_slots, dtype=torch.int32, device="cuda"), S0)
    r = lambda *s: torch.randn(*s, generator=cpu)  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16().cuda()  # noqa: E731
    q, k, v = unit(r(n, H, d)), unit(r(n, H, d)), r(n, H, d).bfloat16().cuda()
    slots = [g.permutation(n_slots)[:n].astype(np.int32) for _ in range(rounds)]
    lens = [(g.random(n) < 0.8).astype(np.int32) for _ in range(rounds)]
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    on_gpu = [(cu(l), cu(s), torch.ones(n, dtype=torch.int32, device="cuda"),
               torch.rand(n, H, generator=cpu).cuda(), torch.rand(n, H, generator=cpu).cuda())
              for l, s in zip(lens, slots)]
    outs = [[torch.zeros(n, H, d, device="cuda") for _ in range(rounds)] for _ in range(2)]
    plan = D.BatchPlan(n, n, n_slots)
    alpha, beta = (torch.zeros(n, H, device="cuda") for _ in range(2))

    def run():
        for (l, s, past, a, b), o in zip(on_gpu, outs[0]):
            alpha.copy_(a)
            beta.copy_(b)
            plan.build(l, s, past)
            pools[0].step(plan.store_slot, q, k, v, alpha, beta, o)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    for i, (l, s) in enumerate(zip(lens, slots)):
        pools[1].step(cu(np.where(l > 0, s, -1).astype(np.int32)), q, k, v, on_gpu[i][3], on_gpu[i][4], outs[1][i])
        torch.cuda.synchronize()
        assert torch.equal(outs[0][i], outs[1][i]), i
    assert torch.equal(pools[0].slots(), pools[1].slots())
    for p in pools:
        assert p.get_error() == 0
        p.close()
