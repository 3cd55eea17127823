"""damp_prefill's bounded waits: a wait that runs out in one part of a kernel ends the whole call with
DAMP_EFLAG_TIMEOUT, and the states stay as they were."""
import numpy as np
import pytest
import torch

import quantized_linear_attention_damp_b200 as D
from tests.prefill_helpers import inputs

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call_under(hooks, rule, lengths, H, fmt="fp32", wait_ns=20_000_000, past=1):
    """One call without the hook (its results), one with it on the same first states, and one more without
    it.  Returns the first states, the states the hook's call left, and the flags it set."""
    d, n, T = 128, len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(T + H)
    x = inputs(g, T, H, H, d, d, BF)
    rows = np.stack([np.arange(h, 64 + h, 3) for h in range(H)]) if fmt == "mixed" else None
    pool = D.DampPool(fmt, n + 1, H, d, rows)
    every = i32(list(range(n + 1)))
    S0 = 0.3 * torch.randn(n + 1, H, d, d, generator=g).cuda()
    slot = torch.randperm(n + 1, generator=g)[:n].tolist()
    plan = D.BatchPlan(n, T, n + 1).build(i32(lengths), i32(slot), i32([past] * n))
    args = (plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"] if rule == "delta" else None)
    # a workspace that holds NaN before each call: nothing of it may reach a state
    need = D.damp_prefill_workspace(pool.handle, D.RULES[rule], n, T, D.DAMP_DTYPE_BF16)
    work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def call():
        work.fill_(255)
        pool.pack(every, S0)
        first = pool.slots().clone()
        out = pool.prefill(*args, rule=rule, workspace=work)
        torch.cuda.synchronize()
        return first, out, pool.slots().clone()

    _, want, states = call()
    assert pool.get_error() == 0
    try:
        D.damp_set_test_hooks(wait_limit_ns=wait_ns, hooks=hooks)
        first, _, after = call()
        flags = pool.get_error(clear=True)
    finally:
        D.damp_set_test_hooks()
    _, again, states2 = call()                            # the context is as good as before
    assert torch.equal(again, want) and torch.equal(states2, states)
    assert pool.get_error() == 0
    pool.close()
    return first, after, flags


@pytest.mark.parametrize("L", [40, 64, 128, 200, 576])
@pytest.mark.parametrize("H", [1, 2, 5])
def test_one_half_of_the_state_warps_runs_out(L, H):
    """Lengths whose first wait of a half is for a ragged block's loads (40), for the only block's product
    (64) and for the first of several (the half that went on is then a block ahead)."""
    first, after, flags = call_under(D.DAMP_HOOK_FAIL_HALF, "delta", [L, 64], H)
    assert flags == D.DAMP_EFLAG_TIMEOUT
    assert torch.equal(after, first)


def test_the_decay_rule_has_no_halves():
    first, after, flags = call_under(D.DAMP_HOOK_FAIL_HALF, "decay", [150, 64], 2)
    assert flags == 0 and not torch.equal(after, first)


@pytest.mark.parametrize("fmt", ["fp32", "mixed"])
@pytest.mark.parametrize("rule,lengths", [("delta", [40, 64, 200]), ("decay", [1200]), ("decay", [2000, 300, 900])])
def test_the_first_of_two_kernels_runs_out(rule, lengths, fmt):
    """The second kernel leaves the states alone when what the first one was to hand over is not there
    (the workspace holds NaN).  The decay rule has two kernels where it cuts requests into segments; the
    one of 300 tokens is a single segment, which does not need the first kernel."""
    H, d, n = 2, 128, len(lengths)
    first, after, flags = call_under(D.DAMP_HOOK_HOLD_FIRST_KERNEL, rule, lengths, H, fmt)
    assert flags == D.DAMP_EFLAG_TIMEOUT
    rows = np.stack([np.arange(h, 64 + h, 3) for h in range(H)]) if fmt == "mixed" else None
    pool = D.DampPool(fmt, n + 1, H, d, rows)
    values = [torch.empty(n + 1, H, d, d, device="cuda") for _ in range(2)]
    for slots, out in zip((first, after), values):
        pool.slots().copy_(slots)
        pool.unpack(i32(list(range(n + 1))), out)
    pool.close()
    # (a quantized pool's values are packed again: half a code's step, 1/127 of the row's largest value)
    step = 0.0 if fmt == "fp32" else values[0].abs().amax(dim=3, keepdim=True) / 127
    kept = ((values[0] - values[1]).abs() <= 0.51 * step).flatten(1).all(dim=1)
    assert torch.isfinite(values[1]).all()
    assert kept.sum() >= n + 1 - (300 in lengths), kept


def test_a_pool_without_tensor_maps():
    """Where the driver's tensor-map encoder cannot be had, only the calls that need it fail."""
    n, H, d, T = 2, 2, 128, 20
    x = inputs(torch.Generator().manual_seed(1), T, H, H, d, d, BF)
    plan = D.BatchPlan(n, T, n).build(i32([15, 5]), i32([1, 0]))
    try:
        D.damp_set_test_hooks(hooks=D.DAMP_HOOK_NO_TENSOR_MAPS)
        pool = D.DampPool("mixed", n, H, d, np.stack([np.arange(27)] * H))
        pool.pack(i32([0, 1]), torch.zeros(n, H, d, d, device="cuda"))
        one = {c: x[c][:n].contiguous() for c in x}
        out = torch.empty(n, H, d, device="cuda")
        pool.step(i32([0, 1]), one["q"], one["k"], one["v"], one["alpha"], one["beta"], out)
        wide = pool.prefill(plan, *(x[c].float() for c in ("q", "k", "v", "alpha", "beta")))
        assert out.any() and wide.any()
        args = (plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"])
        with pytest.raises(D.DampError) as e:
            pool.prefill(*args)
        assert e.value.status == D.DAMP_ERR_CUDA
    finally:
        D.damp_set_test_hooks()
    assert pool.prefill(*args).any() and pool.get_error() == 0
    pool.close()
