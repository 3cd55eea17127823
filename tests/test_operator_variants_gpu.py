"""The forms of the decay-rule step and of the token prefill that only larger batches take.  Each case computes
the rule that chooses its form, so that a change of the rule shows here.  And a refusal of both operators."""
import numpy as np
import pytest
import torch

import oracle as O
import quantized_linear_attention_damp_b200 as D
from tests import test_decay_step_gpu as step
from tests import test_prefill_gpu as prefill
from tests.prefill_helpers import EPS32, decay_step

pytestmark = pytest.mark.gpu

FORMATS = ["fp32", "int8", "mixed", "fp8"]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def warp_per_unit(units, dv):
    return 3 * units >= 2 * 8 * sms() * (3 if dv <= 128 else 2)


def with_padding(n):
    slot = np.random.default_rng(n).permutation(n + 2)[:n].astype(np.int32)
    slot[::7] = -1
    return slot


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dk,dv,n,H,Hqk", [(32, 48, 250, 10, 5), (48, 128, 250, 10, 10), (16, 208, 170, 10, 2),
                                           (16, 256, 164, 10, 1)])
def test_step_with_a_warp_per_state(fmt, dk, dv, n, H, Hqk):
    """All lanes of a warp in use and not, one and two column groups a lane, padding between live entries;
    more states than warps, so that a warp goes on to a next state."""
    assert warp_per_unit(n * H, dv)
    assert step.run(fmt, dk, dv, n, H, Hqk, "bf16", slot_idx=with_padding(n)) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_step_with_a_warp_per_state_and_several_states_a_warp(fmt):
    n, H, dk, dv = 520, 16, 16, 112
    assert n * H > 2 * 3 * 8 * sms()
    assert step.run(fmt, dk, dv, n, H, 8, "f32", steps=1, slot_idx=with_padding(n)) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dk,dv,n,H,Hqk", [(96, 160, 60, 10, 5), (112, 128, 100, 10, 2), (128, 128, 60, 10, 10)])
def test_step_with_a_cta_per_state_and_several_states_a_cta(fmt, dk, dv, n, H, Hqk):
    assert not warp_per_unit(n * H, dv) and n * H > sms() * (3 if dv <= 128 else 2)
    assert step.run(fmt, dk, dv, n, H, Hqk, "bf16", steps=1, slot_idx=with_padding(n)) == 0


@pytest.mark.parametrize("rule", ["decay", "delta"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(16, 144), (32, 16), (48, 80), (64, 64), (96, 48), (128, 112), (208, 16), (256, 48)])
def test_prompts_with_32_rows_a_lane(rule, dtype, dk, dv):
    """Many requests and heads: a lane holds 32 key rows (1, 2, 4 or 8 lanes a column), with padding rows behind
    d_k and column groups that d_v does not fill."""
    n, H = 40, 12
    lanes = 1 if dk <= 32 else 2 if dk <= 64 else 4 if dk <= 128 else 8
    assert n * H * -(-dv * lanes // 128) >= 3 * sms()
    g = np.random.default_rng(dk + dv)
    lengths = g.integers(0, 12, n).tolist()
    lengths[5], lengths[9] = 33, 64
    prefill.check(rule, lengths, H=H, Hqk=4, dk=dk, dv=dv, dtype=dtype, past=g.integers(0, 2, n).tolist(), spare=3)


def test_tensors_on_another_device_than_the_pool_are_refused():
    """(The pool's buffer is only said to lie on another device: nothing is launched.)"""
    class Elsewhere:
        device = torch.device("cuda", 1)

    n, H, d = 2, 2, 128
    pool = D.DampPool("int8", n, H, d)
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    x, gate = torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda"), torch.ones(n, H, device="cuda")
    plan = D.BatchPlan(n, n, n).build(one, torch.arange(n, dtype=torch.int32, device="cuda"))
    mine, pool.buf = pool.buf, Elsewhere
    with pytest.raises(ValueError, match="the pool on cuda:1"):
        pool.prefill(plan, x, x, x, gate, gate)
    with pytest.raises(ValueError, match="the pool on cuda:1"):
        pool.decay_step(one - 1, x, x, x, gate, torch.zeros(n, H, d, device="cuda"))
    pool.buf = mine
    pool.prefill(plan, x, x, x, gate, gate)
    assert pool.get_error() == 0
    pool.close()


@pytest.mark.parametrize("dk,dv,n,H", [(128, 128, 3, 6), (64, 64, 3, 6), (96, 160, 3, 6), (32, 48, 420, 6), (16, 16, 5, 6)])
def test_step_of_pools_whose_heads_differ(dk, dv, n, H):
    """A per-head map: no FP16 row at all, one, all of them, and counts that fill no batch of 8."""
    g = np.random.default_rng(dk)
    counts = [0, 1, dk, dk - 1, dk // 2 + 3, 5]
    is16 = np.zeros((H, dk), np.uint8)
    for h, c in enumerate(counts):
        is16[h, g.permutation(dk)[:c]] = 1
    pool = D.DampPool("mixed", n, H, dk, d_v=dv, fp16_map=is16)
    S0 = g.standard_normal((n, H, dk, dv)).astype(np.float32)
    slot = g.permutation(n).astype(np.int32)
    pool.pack(torch.arange(n, dtype=torch.int32, device="cuda"), torch.from_numpy(S0).cuda())
    st = O.pack(O.FMT_QUANT, is16[None], S0)
    x = [torch.from_numpy(g.standard_normal((n, H, d)).astype(np.float32)).bfloat16() for d in (dk, dk, dv)]
    alpha = g.uniform(0.3, 1.0, (n, H)).astype(np.float32)
    out = torch.empty(n, H, dv, device="cuda")
    pool.decay_step(torch.from_numpy(slot).cuda(), *(t.cuda() for t in x), torch.from_numpy(alpha).cuda(), out)
    got, (q, k, v) = out.cpu().numpy().astype(np.float64), (t.float().numpy() for t in x)
    for b, s in enumerate(slot):
        want, new, X = decay_step(O.FMT_QUANT, is16, st[int(s)], q[b], k[b], v[b], alpha[b])
        for name in ("scale", "half", "code"):
            getattr(st, name)[int(s)] = getattr(new, name)
        # d_k rounded products and sums, each at most half an FP32 step of the running sum
        assert (np.abs(got[b] - want) <= (dk + 2) * EPS32 * (np.abs(q[b])[..., None] * np.abs(X)).sum(axis=-2)).all()
    for name, a in pool.read_logical().items():
        assert np.array_equal(a, getattr(st, name)), name
    assert pool.get_error() == 0
    pool.close()
