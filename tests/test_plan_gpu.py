"""damp_batch_plan against a loop over the requests."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import quantized_linear_attention_damp_b200 as D

pytestmark = pytest.mark.gpu
B = D.DAMP_PLAN_BLOCK


def plain(lengths, past, slot, n_slots, T):
    n = len(lengths)
    cu, load, store, table = [0], [], [], []
    tslot, tpos = np.full(T, -1), np.full(T, -1)
    flags = longest = 0
    total = 0                      # end of the request if none were dropped
    for r in range(n):
        length, p = int(lengths[r]), int(past[r])
        if length < 0 or p < 0:
            flags |= D.DAMP_PLAN_EFLAG_VALUE
        length, p = max(length, 0), max(p, 0)
        if slot[r] >= n_slots:
            flags |= D.DAMP_PLAN_EFLAG_SLOT
        total += length
        if total > T:
            if length:
                flags |= D.DAMP_PLAN_EFLAG_TOKENS
            length = 0
        ok = 0 <= slot[r] < n_slots
        a = cu[-1]
        cu.append(a + length)
        store.append(slot[r] if ok and length else -1)
        load.append(slot[r] if ok and length and p > 0 else -1)
        for i, at in enumerate(range(0, length, B)):
            table.append([r, a + at, min(B, length - at), i])
        tslot[a:a + length] = slot[r] if ok else -1
        tpos[a:a + length] = p + np.arange(length)
        longest = max(longest, length)
    blocks = len(table)
    full = np.full((D.damp_plan_blocks(n, T), 4), -1)
    if blocks:
        full[:blocks] = table
    kept = np.diff(cu)
    order = np.argsort(-kept, kind="stable") if n <= 1024 else np.arange(n)
    return dict(cu_seqlens=cu, load_slot=load, store_slot=store, block_table=full, order=order,
                token_slot=tslot, token_pos=tpos, totals=[cu[-1], blocks, longest, flags])


def check(lengths, past, slot, n_slots, T, token_maps=True):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    p = D.BatchPlan(len(lengths), T, n_slots, token_maps=token_maps)
    for t in (p.cu_seqlens, p.load_slot, p.store_slot, p.block_table, p.order, p.totals, p.token_slot,
              p.token_pos):
        if t is not None:
            t.fill_(12345)
    p.build(i32(lengths), i32(slot), None if past is None else i32(past))
    want = plain(lengths, np.zeros(len(lengths)) if past is None else past, slot, n_slots, T)
    for name, w in want.items():
        got = getattr(p, name)
        if got is None:
            assert not token_maps
            continue
        assert np.array_equal(got.cpu().numpy(), np.asarray(w)), name


@pytest.mark.parametrize("n,top,spare", [(1, 1, 0), (1, 64, 0), (1, 65, 3), (7, 200, 5),
                                         (33, 130, 1), (511, 70, 64), (513, 300, 0),
                                         (5000, 12, 77), (16384, 40, 9)])
def test_ragged(n, top, spare):
    g = np.random.default_rng(n)
    lengths = g.integers(0, top + 1, n)
    if n == 1:
        lengths[0] = top
    slot = g.permutation(n + 2)[:n]
    slot[g.random(n) < 0.1] = -1
    past = np.where(g.random(n) < 0.5, 0, g.integers(1, 1 << 20, n))
    check(lengths, past, slot, n + 2, int(lengths.sum()) + spare)


def test_no_requests_and_no_rows():
    check([], [], [], 4, 0)
    check([], [], [], 4, 70)
    check([0, 0, 0], [5, 0, 1], [2, 1, 0], 4, 9)
    check([0, 0], None, [0, 1], 4, 0)


def test_bad_values_are_counted_as_nothing_and_flagged():
    check([3, -5, 7], [0, 2, -1], [0, 1, 2], 4, 10)
    check([3, 5, 7], None, [0, 99, 2], 4, 20)


def test_requests_that_do_not_fit_are_dropped():
    # the third does not fit; the empty fourth is kept, the short fifth goes with the third
    check([30, 20, 50, 0, 3], [1, 1, 1, 1, 1], [4, 3, 2, 1, 0], 8, 64)
    # sums beyond 2^31 do not wrap
    check([5, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 4], None, [0, 1, 2, 3, 4], 8, 100)


def test_without_past_and_without_token_maps():
    check([10, 0, 129], None, [2, 1, 0], 3, 150, token_maps=False)


def test_captured_build_reads_new_lengths():
    n, T = 6, 500
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lengths, slot = i32([1, 2, 3, 4, 5, 6]), i32([0, 1, 2, 3, 4, 5])
    p = D.BatchPlan(n, T, 8)
    p.build(lengths, slot)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.build(lengths, slot)
    new = [100, 0, 64, 7, 65, 1]
    lengths.copy_(i32(new))
    graph.replay()
    want = plain(new, [0] * n, [0, 1, 2, 3, 4, 5], 8, T)
    for name, w in want.items():
        assert np.array_equal(getattr(p, name).cpu().numpy(), np.asarray(w)), name


def test_first_build_of_a_process_with_many_requests():
    """Offsets of 5,600 to 6,144 requests, with the kernel's own shared memory, just pass the 48 KB that a
    launch has without asking for more; a larger build before would have asked already."""
    code = """
import torch, quantized_linear_attention_damp_b200 as D
one = torch.ones(6144, dtype=torch.int32, device="cuda")
for n in (5000, 5600, 6000, 6144):
    p = D.BatchPlan(n, n, 1).build(one[:n], torch.zeros_like(one[:n]))
    assert p.totals.tolist() == [n, n, 1, 0], (n, p.totals)
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=Path(__file__).resolve().parent.parent)
