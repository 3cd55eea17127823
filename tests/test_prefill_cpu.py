"""Refusals of the plan, decay-step and prefill calls (no kernel is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_linear_attention_damp_b200 as D

INV, UNS, MIS, SMALL = (D.DAMP_ERR_INVALID_ARGUMENT, D.DAMP_ERR_UNSUPPORTED, D.DAMP_ERR_MISALIGNED,
                        D.DAMP_ERR_BUFFER_TOO_SMALL)
lib = D._lib
P16 = ctypes.c_void_p(4096)      # an aligned address that no call may read
ODD = ctypes.c_void_p(4104)


@pytest.fixture
def host_pool():
    h = D.damp_pool_create(D.DAMP_FMT_FP32, 4, 6, 128, 128, 0, None, None)
    yield h
    D.damp_pool_destroy(h)


def test_plan_block_counts():
    assert D.damp_plan_blocks(0, 0) == 0
    assert D.damp_plan_blocks(1, 1) == 1
    assert D.damp_plan_blocks(1, 65) == 2
    assert D.damp_plan_blocks(3, 3) == 3
    # the bound holds for the raggedest lengths: Sum ceil(L / 64) <= (T + 63 n) / 64
    g = np.random.default_rng(0)
    for _ in range(200):
        n = int(g.integers(1, 30))
        lengths = g.integers(0, 200, n)
        assert -(-lengths // 64).sum() <= D.damp_plan_blocks(n, int(lengths.sum()))
    out = ctypes.c_int()
    assert lib.damp_plan_blocks(-1, 0, ctypes.byref(out)) == INV
    assert lib.damp_plan_blocks(1, -1, ctypes.byref(out)) == INV
    assert lib.damp_plan_blocks(1, 1, None) == INV
    assert lib.damp_plan_blocks(D.DAMP_PLAN_MAX_REQUESTS + 1, 1, ctypes.byref(out)) == UNS
    assert lib.damp_plan_blocks(1, D.DAMP_PLAN_MAX_TOKENS + 1, ctypes.byref(out)) == UNS


def plan_args(**kw):
    a = dict(n=2, lengths=P16, past=None, slot_idx=P16, n_slots=4, max_tokens=100, cu=P16, load=P16,
             store=P16, table=P16, tslot=P16, tpos=P16, order=None, totals=P16, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INV), (dict(max_tokens=-1), INV), (dict(n_slots=0), INV), (dict(lengths=None), INV),
    (dict(slot_idx=None), INV), (dict(cu=None), INV), (dict(load=None), INV), (dict(store=None), INV),
    (dict(table=None), INV), (dict(totals=None), INV), (dict(tslot=None), INV), (dict(tpos=None), INV),
    (dict(table=ODD), MIS), (dict(tslot=ODD), MIS), (dict(tpos=ODD), MIS),
    (dict(lengths=ctypes.c_void_p(4098)), MIS), (dict(order=ctypes.c_void_p(4097)), MIS), (dict(n=D.DAMP_PLAN_MAX_REQUESTS + 1), UNS)])
def test_plan_refuses(kw, rc):
    assert lib.damp_batch_plan(*plan_args(**kw)) == rc


def step_args(pool, **kw):
    a = dict(pool=pool, n=2, slot=P16, dt=0, hqk=3, q=P16, k=P16, v=P16, alpha=P16, out=P16, stream=None)
    a.update(kw)
    return list(a.values())


def test_decay_step_refuses(host_pool):
    assert lib.damp_decay_step(*step_args(None)) == INV
    assert lib.damp_decay_step(*step_args(host_pool)) == INV          # a host-only descriptor


def prefill_args(pool, **kw):
    a = dict(pool=pool, rule=0, n=2, T=10, cu=P16, load=P16, store=P16, table=P16, order=None, dt=0, hqk=3, q=P16,
             qs=384, k=P16, ks=384, v=P16, vs=768, alpha=P16, beta=P16, out=P16, ws=P16, wsb=1 << 40,
             stream=None)
    a.update(kw)
    return list(a.values())


def test_prefill_refuses(host_pool):
    assert lib.damp_prefill(*prefill_args(None)) == INV
    assert lib.damp_prefill(*prefill_args(host_pool)) == INV          # a host-only descriptor
    for kw, rc in ((dict(rule=2), INV), (dict(rule=-1), INV), (dict(n=-1), INV), (dict(T=-1), INV),
                   (dict(dt=2), INV), (dict(n=D.DAMP_PLAN_MAX_REQUESTS + 1), UNS),
                   (dict(T=D.DAMP_PLAN_MAX_TOKENS + 1), UNS)):
        assert lib.damp_prefill(*prefill_args(host_pool, **kw)) == rc, kw


def test_workspace_sizes(host_pool):
    w = ctypes.c_size_t()
    assert lib.damp_prefill_workspace(host_pool, 0, 2, 10, 0, None) == INV
    assert lib.damp_prefill_workspace(host_pool, 5, 2, 10, 0, ctypes.byref(w)) == INV
    assert lib.damp_prefill_workspace(None, 0, 2, 10, 0, ctypes.byref(w)) == INV
    q = D.damp_pool_create(D.DAMP_FMT_INT8_ROW, 4, 6, 64, 32, 0, None, None)
    # FP32 states of the batch for a pool whose blocks are quantized
    assert D.damp_prefill_workspace(q, 0, 3, 10, 1) >= 3 * 6 * 64 * 32 * 4
    D.damp_pool_destroy(q)


def test_binding_refuses_host_tensors_and_wrong_shapes(host_pool):
    z = torch.zeros
    i = lambda n: z(n, dtype=torch.int32)  # noqa: E731
    q, v = z(5, 3, 128), z(5, 6, 128)
    good = dict(slot_idx=i(5), q=q, k=q, v=v, alpha=z(5, 6), out=z(5, 6, 128))
    for bad in (dict(), dict(q=z(5, 4, 128)), dict(q=z(5, 128)), dict(k=z(5, 6, 128)),
                dict(v=z(5, 6, 64)), dict(alpha=z(5, 6, 128)), dict(out=z(4, 6, 128)),
                dict(slot_idx=i((5, 1)))):
        with pytest.raises(ValueError):
            D.damp_decay_step(host_pool, **{**good, **bad})
    pre = dict(rule=0, cu_seqlens=i(3), load_slot=i(2), store_slot=i(2),
               block_table=i((D.damp_plan_blocks(2, 5), 4)), order=None, q=q, k=q, v=v, alpha=z(5, 6),
               beta=z(5, 6), out=z(5, 6, 128))
    for bad in (dict(), dict(rule=7), dict(q=z(5, 4, 128)), dict(v=z(5, 5, 128)),
                dict(beta=None), dict(rule=1), dict(alpha=z(5, 3)), dict(cu_seqlens=i(2))):
        with pytest.raises(ValueError):
            D.damp_prefill(host_pool, **{**pre, **bad})
    with pytest.raises(ValueError):
        D.damp_batch_plan(i(2), i(2), None, 4, 10, i(3), i(2), i(2), i((2, 4)), None, None, None, i(4))
    with pytest.raises(ValueError):
        D.damp_batch_plan(i((2, 1)), i(2), None, 4, 10, i(3), i(2), i(2), i((2, 4)), None, None, None, i(4))


def test_token_rows_must_be_dense_inside():
    t = torch.zeros(4, 6, 32)
    assert D._token_stride(t, "q") == 192
    assert D._token_stride(t[::2], "q") == 384
    assert D._token_stride(t[:, :3], "q") == 192
    assert D._token_stride(t[:1], "q") == 192
    assert D._token_stride(t[:, :1], "q") == 192
    for bad in (t[:, ::2], t[..., ::2], t.transpose(0, 1)):
        with pytest.raises(ValueError):
            D._token_stride(bad, "q")
