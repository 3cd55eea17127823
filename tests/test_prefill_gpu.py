"""damp_prefill against the token recurrence in 64 bits."""
import threading

import numpy as np
import pytest
import torch

import quantized_linear_attention_damp_b200 as D
from tests.prefill_helpers import EPS32, EPS_BF16, inputs, recurrence

pytestmark = pytest.mark.gpu

# Bound of one state (Frobenius norm), relative to the largest state or update on the way.
#   token kernels: every token rounds a state value at most 3 times and the projection k^T S sums
#     d_k products, all in FP32: (3 L + d_k) half steps.
#   chunk kernels: an FP32 operand of a matrix product is split into bf16 pairs, which leaves at
#     most 2^-17 of it; at most 8 such splits lie between the inputs and a state.  The products'
#     FP32 sums add less than the token kernels' bound.
SPLITS = 8 * 2.0 ** -17


def tolerance(L, dk, chunked):
    return (3 * L + dk) * EPS32 + (SPLITS if chunked else 0.0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(rule, lengths, H, Hqk, dk, dv, dtype, fmt="fp32", past=None, slot=None, spare=0, edit=None,
          strided=False, seed=0, n_slots=None, stream=None, runs=1, device="cuda"):
    """One call on fresh states, compared request by request; rows and slots that no request owns
    have to keep what they held."""
    n, T = len(lengths), sum(lengths) + spare
    g = torch.Generator().manual_seed(seed + 17 * T + dk)
    x = inputs(g, T, H, Hqk, dk, dv, dtype)
    if edit:
        edit(x)
    n_slots = n + 2 if n_slots is None else n_slots
    slot = list(torch.randperm(n_slots, generator=g)[:n].tolist()) if slot is None else slot
    past = [0] * n if past is None else past
    S0 = 0.3 * torch.randn(n_slots, H, dk, dv, generator=g).cuda()
    hp = dk // 4
    rows = np.stack([np.sort(np.random.default_rng(h).permutation(dk)[:hp]) for h in range(H)])
    pool = D.DampPool(fmt, n_slots, H, dk, rows if fmt == "mixed" else None, d_v=dv)
    every = i32(list(range(n_slots)))
    pool.pack(every, S0)
    pool.unpack(every, S0)                     # what the pool holds
    before = pool.slots().clone()
    plan = D.BatchPlan(n, T, n_slots).build(i32(lengths), i32(slot), i32(past))
    if strided:                                # q, k, v as columns of one projection's output
        width = 2 * Hqk * dk + H * dv
        wide = torch.zeros(T, width + 16, dtype=dtype, device="cuda")
        q = wide[:, :Hqk * dk].view(T, Hqk, dk)
        k = wide[:, Hqk * dk:2 * Hqk * dk].view(T, Hqk, dk)
        v = wide[:, 2 * Hqk * dk:width].view(T, H, dv)
        q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    else:
        q, k, v = x["q"], x["k"], x["v"]
    out = torch.full((T, H, dv), 5.0, dtype=dtype, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    pool.prefill(plan, q, k, v, x["alpha"], x["beta"] if rule == "delta" else None, out, rule=rule,
                 stream=stream)
    torch.cuda.synchronize()
    chunked = dtype == torch.bfloat16 and dk == dv == 128
    S1 = torch.empty_like(S0)
    pool.unpack(every, S1)
    after = pool.slots()
    at, touched = 0, set()
    for r, L in enumerate(lengths):
        a, at = at, at + L
        if not 0 <= slot[r] < n_slots:
            assert not out[a:at].any()
            continue
        if L == 0:
            continue
        touched.add(slot[r])
        S = S0[slot[r]] if past[r] > 0 else torch.zeros_like(S0[0])
        o, S, top = recurrence(rule, *(x[c][a:at] for c in ("q", "k", "v", "alpha", "beta")), S)
        tol = tolerance(L, dk, chunked) * top                              # [H]
        err = (S1[slot[r]].double() - S).flatten(1).norm(dim=1)
        room = tol
        if fmt != "fp32":
            # the pool's own rounding: half an INT8 step of each row's largest value (FP16 rows and
            # the FP32 roundings of the scale are far below it), or 2^-4 of each value
            step = S.abs().amax(dim=2) / 127 * 0.5 * dv ** 0.5
            room = room + (step.norm(dim=1) if fmt != "fp8" else 2.0 ** -4 * S.flatten(1).norm(dim=1)) * 1.01
        assert (err <= room).all(), (r, (err / room).max())
        qn = x["q"][a:at].double().norm(dim=-1).repeat_interleave(H // Hqk, dim=1)
        half = EPS_BF16 if dtype == torch.bfloat16 else EPS32
        got = out[a:at].double()
        lim = half * o.abs() + ((tol + dk * EPS32 * top)[None] * qn)[..., None]
        assert ((got - o).abs() <= lim).all(), (r, ((got - o).abs() / lim).max())
    assert (out[sum(lengths):] == 5.0).all()
    for s in range(n_slots):
        if s not in touched:
            assert torch.equal(after[s], before[s]), s
    err = pool.get_error()
    pool.close()
    return err


RULES = ["decay", "delta"]
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 64), (48, 208), (256, 32), (128, 128), (160, 128)])
def test_shapes(rule, dtype, dk, dv):
    check(rule, [5, 1, 33, 0, 70], H=4, Hqk=2, dk=dk, dv=dv, dtype=dtype, past=[0, 3, 0, 1, 9],
          spare=6)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("L", [1, 2, 15, 63, 64, 65, 127, 128, 129, 192, 300])
def test_lengths_at_block_edges(rule, L):
    check(rule, [L], H=2, Hqk=1, dk=128, dv=128, dtype=BF, past=[L % 2])
    check(rule, [3, L, 1], H=1, Hqk=1, dk=128, dv=128, dtype=BF, past=[0, 1, 1], spare=1)


@pytest.mark.parametrize("rule", RULES)
def test_long_request(rule):
    check(rule, [1111, 40], H=2, Hqk=2, dk=128, dv=128, dtype=BF, past=[1, 0])


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_one_projection(rule, dtype):
    check(rule, [70, 9, 130], H=4, Hqk=2, dk=128, dv=128, dtype=dtype, strided=True, spare=3)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("fmt", ["int8", "mixed", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_quantized_pools(rule, fmt, d):
    check(rule, [20, 0, 90, 5], H=3, Hqk=3, dk=d, dv=d, dtype=BF, fmt=fmt, past=[4, 7, 0, 1], spare=2)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_entries_and_bad_slots(rule, dtype):
    # the plan turns a slot out of range into padding
    check(rule, [10, 80, 7], H=2, Hqk=2, dk=128, dv=128, dtype=dtype, slot=[-1, 1, 50], past=[1, 1, 1])


def test_slot_out_of_range_in_the_arrays_is_flagged():
    H = d = 128
    H = 2
    T = 12
    for dtype in (BF, F32):
        x = inputs(torch.Generator().manual_seed(1), T, H, H, d, d, dtype)
        pool = D.DampPool("fp32", 3, H, d)
        pool.slots().fill_(0)
        plan = D.BatchPlan(2, T, 3).build(i32([5, 7]), i32([0, 1]))
        plan.store_slot[1] = 9
        out = pool.prefill(plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"])
        assert pool.get_error() == D.DAMP_EFLAG_SLOT_RANGE
        assert out[:5].any() and not out[5:].any()
        assert not pool.slots()[1:].any()
        pool.close()


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_and_absent_decay(rule, dtype):
    def edit(x):
        a = x["alpha"]
        a[:20] = 1.0
        a[20:40] = 1e-6
        a[60] = 0.0                        # forgets everything before
        a[61] = 0.0
        a[100:180] = 0.0
        a[190:] = 0.5
        x["beta"][30:50] = 1.0
        x["beta"][50:55] = 0.0

    check(rule, [230, 31], H=2, Hqk=2, dk=128, dv=128, dtype=dtype, past=[1, 0], edit=edit)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_keys(dtype):
    """Every key of a block the same: the triangular system is at its worst (all of A is beta)."""
    def edit(x):
        x["k"][:] = x["k"][:1]
        x["alpha"][:] = 1.0

    check("delta", [150], H=2, Hqk=2, dk=128, dv=128, dtype=dtype, edit=edit)


@pytest.mark.parametrize("rule", RULES)
def test_on_another_stream(rule):
    check(rule, [70, 5], H=2, Hqk=2, dk=128, dv=128, dtype=BF, stream=torch.cuda.Stream())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("fmt", ["fp32", "mixed"])
def test_captured_calls_match_eager_ones(rule, fmt):
    """A plan and two layers captured, replayed on new lengths and inputs; workspaces of the two
    layers are their own."""
    H, d, n, T = 2, 128, 3, 200
    rows = np.stack([np.arange(20) for _ in range(H)])
    mk = lambda: D.DampPool(fmt, 4, H, d, rows if fmt == "mixed" else None)  # noqa: E731
    pools = [[mk(), mk()] for _ in range(2)]
    S0 = torch.randn(4, H, d, d, generator=torch.Generator().manual_seed(1)).cuda()
    for pair in pools:
        for p in pair:
            p.pack(i32([0, 1, 2, 3]), S0)
    lengths, slot, past = i32([0, 0, 0]), i32([2, 0, 3]), i32([1, 0, 1])
    x = inputs(torch.Generator().manual_seed(2), T, H, H, d, d, BF)
    outs = [[torch.zeros(T, H, d, dtype=BF, device="cuda") for _ in range(2)] for _ in range(2)]
    plan = D.BatchPlan(n, T, 4)

    def layers(i):
        plan.build(lengths, slot, past)
        for p, o in zip(pools[i], outs[i]):
            p.prefill(plan, x["q"], x["k"], x["v"], x["alpha"],
                      x["beta"] if rule == "delta" else None, o, rule=rule)

    layers(1)                               # lengths of zero: nothing may change
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers(1)
    for new in ([70, 3, 100], [1, 0, 199]):
        lengths.copy_(i32(new))
        x["v"].add_(0.25)
        graph.replay()
        layers(0)
        torch.cuda.synchronize()
        for l in range(2):
            assert torch.equal(outs[0][l], outs[1][l])
            assert torch.equal(pools[0][l].slots(), pools[1][l].slots())


@pytest.mark.parametrize("rule", RULES)
def test_same_inputs_same_bits(rule):
    x = inputs(torch.Generator().manual_seed(5), 300, 4, 4, 128, 128, BF)
    got = []
    for _ in range(2):
        pool = D.DampPool("fp32", 2, 4, 128)
        pool.slots().fill_(0)
        plan = D.BatchPlan(2, 300, 2).build(i32([260, 40]), i32([1, 0]))
        o = pool.prefill(plan, x["q"], x["k"], x["v"], x["alpha"],
                         x["beta"] if rule == "delta" else None, rule=rule)
        got.append((o.clone(), pool.slots().clone()))
        pool.close()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("rule", RULES)
def test_prompt_then_single_tokens(rule):
    """The operators as they are used: plan, prefill, then steps that go on from the pool's
    states, against one recurrence over all tokens."""
    H, d, L, more = 3, 128, 100, 6
    g = torch.Generator().manual_seed(9)
    x = inputs(g, L + more, H, H, d, d, BF)
    pool = D.DampPool("fp32", 2, H, d)
    plan = D.BatchPlan(1, L, 2).build(i32([L]), i32([1]))
    out = pool.prefill(plan, x["q"][:L], x["k"][:L], x["v"][:L], x["alpha"][:L],
                       x["beta"][:L] if rule == "delta" else None, rule=rule)
    rows = [out.double()]
    for t in range(L, L + more):
        o = torch.empty(1, H, d, device="cuda")
        s = {c: x[c][t:t + 1].contiguous() for c in x}
        if rule == "delta":
            pool.step(i32([1]), s["q"], s["k"], s["v"], s["alpha"], s["beta"], o)
        else:
            pool.decay_step(i32([1]), s["q"], s["k"], s["v"], s["alpha"], o)
        rows.append(o.double())
    want, S, top = recurrence(rule, x["q"], x["k"], x["v"], x["alpha"], x["beta"],
                              torch.zeros(H, d, d, device="cuda"))
    tol = tolerance(L + more, d, True) * top
    got = torch.cat(rows)
    assert ((got - want).abs() <= EPS_BF16 * want.abs() + tol[None, :, None] * 1.01).all()
    S1 = torch.empty(1, H, d, d, device="cuda")
    pool.unpack(i32([1]), S1)
    assert ((S1[0].double() - S).flatten(1).norm(dim=1) <= tol).all()
    pool.close()


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_request_does_not_see_its_neighbours(rule, dtype, bad):
    """Requests 1 and 3 and the rows behind the last hold NaN or infinities; blocks of the others
    end inside the same 64-row tiles."""
    H, d, lengths = 2, 128, [70, 5, 30, 90, 1, 64]
    T = sum(lengths) + 80
    x = inputs(torch.Generator().manual_seed(4), T, H, H, d, d, dtype)
    at = np.concatenate([[0], np.cumsum(lengths)])

    def run(x):
        pool = D.DampPool("fp32", 6, H, d)
        pool.slots().fill_(0)
        plan = D.BatchPlan(6, T, 6).build(i32(lengths), i32([0, 1, 2, 3, 4, 5]))
        o = pool.prefill(plan, x["q"], x["k"], x["v"], x["alpha"],
                         x["beta"] if rule == "delta" else None, rule=rule)
        s = pool.slots().clone()
        pool.close()
        return o, s

    o0, s0 = run(x)
    y = {k: v.clone() for k, v in x.items()}
    for r in (1, 3, 6):
        a, b = (at[r], at[r + 1]) if r < 6 else (at[6], T)
        for c in ("q", "k", "v", "alpha", "beta"):
            y[c][a:b] = bad
    o1, s1 = run(y)
    for r in (0, 2, 4, 5):
        assert torch.equal(o0[at[r]:at[r + 1]], o1[at[r]:at[r + 1]]), r
        assert torch.equal(s0[r], s1[r]), r


@pytest.mark.parametrize("rule", RULES)
def test_a_wait_that_runs_out_is_reported(rule):
    H, d, T = 3, 128, 150
    x = inputs(torch.Generator().manual_seed(4), T, H, H, d, d, BF)
    pool = D.DampPool("fp32", 3, H, d)
    pool.slots().fill_(0)
    plan = D.BatchPlan(2, T, 3).build(i32([100, 50]), i32([2, 0]), i32([1, 1]))
    args = (plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"] if rule == "delta" else None)
    want = pool.prefill(*args, rule=rule)
    states = pool.slots().clone()
    pool.slots().fill_(0)
    try:
        D.damp_set_test_hooks(wait_limit_ns=3_000_000, hooks=D.DAMP_HOOK_HOLD_FIRST_ITEM)
        pool.prefill(*args, rule=rule)
        assert pool.get_error(clear=True) == D.DAMP_EFLAG_TIMEOUT
        assert not pool.slots().any()
    finally:
        D.damp_set_test_hooks()
    assert torch.equal(pool.prefill(*args, rule=rule), want)      # the context is as good as before
    assert torch.equal(pool.slots(), states)
    assert pool.get_error() == 0
    pool.close()


@pytest.mark.parametrize("rule", RULES)
def test_many_short_requests_and_few_heads(rule):
    g = np.random.default_rng(1)
    lengths = g.integers(0, 9, 200).tolist()
    check(rule, lengths, H=1, Hqk=1, dk=128, dv=128, dtype=BF, past=g.integers(0, 2, 200).tolist())


def test_segments_of_long_requests():
    """The decay rule cuts requests into segments where few chains would leave SMs idle; ragged
    lengths give empty and short segments, and the first and the last one share a slot."""
    for lengths in ([2048, 300, 5, 0, 64], [4000], [257, 1, 1900]):
        check("decay", lengths, H=1, Hqk=1, dk=128, dv=128, dtype=BF, past=[1] * len(lengths), spare=7)
        check("decay", lengths, H=2, Hqk=1, dk=128, dv=128, dtype=BF, past=[0] * len(lengths))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_offsets_past_32_bits(rule, dtype, d):
    """A request behind 4 GiB of token rows, its state behind 4 GiB of slots."""
    H, first, L = 128, 1 << 17, 70
    n_slots = (1 << 32) // (H * d * d * 4) + 2
    g = torch.Generator().manual_seed(d)
    x = inputs(g, L, H, 2, d, d, dtype)

    def behind(t):
        big = torch.zeros(first + L, *t.shape[1:], dtype=t.dtype, device="cuda")
        big[first:] = t
        return big

    pool = D.DampPool("fp32", n_slots, H, d)
    S0 = 0.3 * torch.randn(H, d, d, generator=g).cuda()
    pool.pack(i32([n_slots - 1]), S0[None])
    plan = D.BatchPlan(2, first + L, n_slots).build(i32([first, L]), i32([-1, n_slots - 1]), i32([0, 1]))
    out = torch.ones(first + L, H, d, dtype=dtype, device="cuda")
    pool.prefill(plan, behind(x["q"]), behind(x["k"]), behind(x["v"]), behind(x["alpha"]),
                 behind(x["beta"]) if rule == "delta" else None, out, rule=rule)
    assert not out[:64].any() and not out[first - 64:first].any()
    o, S, top = recurrence(rule, x["q"], x["k"], x["v"], x["alpha"], x["beta"], S0)
    S1 = torch.empty(1, H, d, d, device="cuda")
    pool.unpack(i32([n_slots - 1]), S1)
    tol = tolerance(L, d, dtype == BF) * top
    assert ((S1[0].double() - S).flatten(1).norm(dim=1) <= tol).all()
    qn = x["q"].double().norm(dim=-1).repeat_interleave(H // 2, dim=1)
    lim = (EPS_BF16 if dtype == BF else EPS32) * o.abs() + ((tol + d * EPS32 * top)[None] * qn)[..., None]
    assert ((out[first:].double() - o).abs() <= lim).all()
    assert pool.get_error() == 0
    pool.close()


@pytest.mark.parametrize("rule", RULES)
def test_two_calls_at_once(rule):
    """Two layers on two streams at the same time, each with its own pool and workspace."""
    H, d, T = 4, 128, 700
    x = inputs(torch.Generator().manual_seed(8), T, H, H, d, d, BF)
    plan = D.BatchPlan(3, T, 3).build(i32([300, 250, 150]), i32([2, 0, 1]))
    pools = [D.DampPool("fp32", 3, H, d) for _ in range(3)]
    for p in pools:
        p.slots().fill_(0)
    args = (plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"] if rule == "delta" else None)
    want = pools[0].prefill(*args, rule=rule)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s, o in zip(pools[1:], streams, outs):
            p.prefill(*args, o, rule=rule, stream=s)
    torch.cuda.synchronize()
    for p, o in zip(pools[1:], outs):
        assert torch.equal(o, want) and torch.equal(p.slots(), pools[0].slots())


@pytest.mark.parametrize("what", ["prefill", "step"])
def test_two_host_threads(what):
    """Two threads launch the same kernel with different amounts of shared memory."""
    errors, start = [], threading.Barrier(2)

    def run(d_k, dtype):
        try:
            g = torch.Generator().manual_seed(d_k)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                pool = D.DampPool("fp32", 2, 2, d_k, d_v=48)
                pool.slots().fill_(0)
                x = inputs(g, 2, 2, 2, d_k, 48, dtype)
                plan = D.BatchPlan(2, 2, 2).build(i32([1, 1]), i32([1, 0]))
                out = torch.empty(2, 2, 48, device="cuda")
            start.wait()
            for _ in range(400):
                if what == "prefill":
                    pool.prefill(plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"], stream=stream)
                else:
                    pool.decay_step(plan.store_slot, x["q"], x["k"], x["v"], x["alpha"], out, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=a) for a in ((144, BF), (256, torch.float32))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_refusals_with_a_device_pool():
    H, d, T = 2, 128, 8
    x = inputs(torch.Generator().manual_seed(1), T, H, H, d, d, BF)
    pool = D.DampPool("mixed", 3, H, d, np.array([[0, 5], [7, 9]]))
    plan = D.BatchPlan(1, T, 3).build(i32([T]), i32([0]))
    ok = dict(plan=plan, q=x["q"], k=x["k"], v=x["v"], alpha=x["alpha"], beta=x["beta"])
    for bad in (dict(q=x["q"].float()), dict(k=x["k"].float()), dict(beta=None), dict(rule="decay"),
                dict(alpha=x["alpha"].half()), dict(alpha=x["alpha"][:, :1]),
                dict(q=x["q"][..., ::2]), dict(plan=D.BatchPlan(1, T, 4)), dict(plan=D.BatchPlan(1, T + 1, 3)),
                dict(out=torch.zeros(T, H, d, device="cuda")), dict(rule="gated")):
        with pytest.raises((ValueError, KeyError)):
            pool.prefill(**{**ok, **bad})
    with pytest.raises(ValueError, match="not been built"):
        pool.prefill(**{**ok, "plan": D.BatchPlan(1, T, 3)})
    need = D.damp_prefill_workspace(pool.handle, D.DAMP_RULE_DELTA, 1, T, D.DAMP_DTYPE_BF16)
    with pytest.raises(D.DampError) as e:
        pool.prefill(**ok, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == D.DAMP_ERR_BUFFER_TOO_SMALL
    with pytest.raises(D.DampError) as e:
        pool.prefill(**ok, workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:])
    assert e.value.status == D.DAMP_ERR_MISALIGNED
    odd = torch.zeros(T, H * d + 4, dtype=BF, device="cuda")[:, :H * d].view(T, H, d)
    with pytest.raises(D.DampError) as e:                          # rows not 16 bytes apart
        pool.prefill(**{**ok, "v": odd})
    assert e.value.status == D.DAMP_ERR_MISALIGNED
    with pytest.raises(D.DampError) as e:                          # every row the same one
        pool.prefill(**{**ok, "v": x["v"][:1].expand(T, H, d)})
    assert e.value.status == D.DAMP_ERR_INVALID_ARGUMENT
    pool.prefill(**ok, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert pool.get_error() == 0
    pool.close()
