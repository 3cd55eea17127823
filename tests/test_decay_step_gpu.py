"""damp_decay_step: states bit for bit, readouts against 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import quantized_linear_attention_damp_b200 as D
from tests.gpu_helpers import oracle_fmt
from tests.prefill_helpers import EPS32, decay_step

pytestmark = pytest.mark.gpu


def run(fmt, dk, dv, n, H, Hqk, dtype, steps=2, slot_idx=None, edit=None):
    g = np.random.default_rng([dk, dv, n, H, Hqk])
    n_slots = n + 2
    hp = 0 if fmt != "mixed" else max(1, dk // 5)
    is16 = np.zeros((H, dk), np.uint8)
    for h in range(H):
        is16[h, g.permutation(dk)[:hp]] = 1
    rows = np.stack([np.flatnonzero(m) for m in is16]) if hp else None
    S0 = (g.standard_normal((n_slots, H, dk, dv)) * np.exp(g.standard_normal((n_slots, H, dk, 1)))
          ).astype(np.float32)
    S0[0, 0, 1] = 0.0                       # a zero row
    pool = D.DampPool(fmt, n_slots, H, dk, rows, d_v=dv)
    pool.pack(torch.arange(n_slots, dtype=torch.int32, device="cuda"), torch.from_numpy(S0).cuda())
    ofmt = oracle_fmt(fmt)
    st = O.pack(ofmt, is16[None], S0)
    if slot_idx is None:
        slot_idx = g.permutation(n_slots)[:n].astype(np.int32)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    for s in range(steps):
        x = {name: torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(td)
             for name, shape in (("q", (n, Hqk, dk)), ("k", (n, Hqk, dk)), ("v", (n, H, dv)))}
        alpha = g.uniform(0.3, 1.0, (n, H)).astype(np.float32)
        if edit:
            edit(x, alpha)
        out = torch.full((n, H, dv), 7.0, device="cuda")
        pool.decay_step(torch.from_numpy(slot_idx).cuda(), *(x[c].cuda() for c in "qkv"),
                        torch.from_numpy(alpha).cuda(), out)
        f = {c: x[c].float().numpy() for c in "qkv"}
        f["q"], f["k"] = (np.repeat(f[c], H // Hqk, axis=1) for c in "qk")
        got = out.cpu().numpy().astype(np.float64)
        for b, slot in enumerate(slot_idx):
            if not 0 <= slot < n_slots:
                assert not got[b].any()
                continue
            want, new, X = decay_step(ofmt, is16, st[int(slot)], f["q"][b], f["k"][b], f["v"][b],
                                      alpha[b])
            for name in ("scale", "half", "code", "f32"):
                old = getattr(st, name, None)
                if old is not None:
                    old[int(slot)] = getattr(new, name)
            # d_k rounded products and sums, each at most half an FP32 step of the running sum
            bound = (dk + 2) * EPS32 * (np.abs(f["q"][b])[..., None] * np.abs(X)).sum(axis=-2)
            assert (np.abs(got[b] - want) <= bound + 1e-30).all()
        lg = pool.read_logical()
        for name, a in lg.items():
            assert np.array_equal(a, getattr(st, name)), (name, s)
    err = pool.get_error()
    pool.close()
    return err


@pytest.mark.parametrize("fmt", ["fp32", "int8", "mixed", "fp8"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 32), (64, 64), (128, 128), (96, 160), (256, 16),
                                   (16, 240)])
def test_formats_and_shapes(fmt, dk, dv):
    assert run(fmt, dk, dv, n=3, H=4, Hqk=2, dtype="bf16") == 0


@pytest.mark.parametrize("n,H,Hqk", [(1, 1, 1), (5, 3, 3), (2, 7, 1), (9, 6, 2)])
def test_batches_and_shared_heads_fp32_inputs(n, H, Hqk):
    assert run("mixed", 128, 128, n, H, Hqk, "f32") == 0
    assert run("int8", 32, 32, n, H, Hqk, "f32") == 0


@pytest.mark.parametrize("d", [64, 128, 48])
def test_padding_and_slots_out_of_range(d):
    err = run("mixed", d, d, n=4, H=2, Hqk=2, dtype="bf16",
              slot_idx=np.array([2, -1, 77, 0], np.int32))
    assert err == D.DAMP_EFLAG_SLOT_RANGE


@pytest.mark.parametrize("fmt", ["fp32", "mixed"])
def test_forgetting_and_empty_updates(fmt):
    def edit(x, alpha):
        alpha[0] = 0.0                      # only this token's k v^T is left
        x["k"][1] = 0                       # pure decay
        x["v"][2] = 0

    assert run(fmt, 128, 128, n=4, H=2, Hqk=1, dtype="bf16", edit=edit) == 0


def test_captured_steps_on_another_stream():
    n, H, d = 4, 2, 128
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    q, k, v = (mk(n, H, d).bfloat16() for _ in range(3))
    alpha = torch.rand(n, H, generator=g).cuda()
    slot = torch.arange(n, dtype=torch.int32, device="cuda")
    S0 = mk(n, H, d, d)
    pools = [D.DampPool("int8", n, H, d) for _ in range(2)]
    outs = [torch.empty(n, H, d, device="cuda") for _ in range(2)]
    for p in pools:
        p.pack(slot, S0)
    for _ in range(3):
        pools[0].decay_step(slot, q, k, v, alpha, outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pools[1].decay_step(slot, q, k, v, alpha, outs[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            graph.replay()
    pools[1].decay_step(slot, q, k, v, alpha, outs[1], stream=side)
    side.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(pools[0].slots(), pools[1].slots())


@pytest.mark.parametrize("fmt", ["fp32", "mixed", "fp8"])
def test_slots_past_32_bits(fmt):
    """Slots behind 4 GiB of others give bit for bit what a small pool gives (5120 states, a warp each,
    and 256, a CTA each)."""
    H, d = 128, 128
    g = torch.Generator().manual_seed(3)
    rows = np.stack([np.arange(h % 4, 108, 4) for h in range(H)]) if fmt == "mixed" else None
    for n in (40, 2):
        small = D.DampPool(fmt, n, H, d, rows)
        n_slots = (1 << 32) // (small.nbytes // n) + n + 2
        big = D.DampPool(fmt, n_slots, H, d, rows)
        S0 = torch.randn(n, H, d, d, generator=g).cuda()
        at = [torch.arange(a, a + n, dtype=torch.int32, device="cuda") for a in (0, n_slots - n)]
        x = [torch.randn(n, H, d, generator=g).bfloat16().cuda() for _ in range(3)]
        alpha = torch.rand(n, H, generator=g).cuda()
        out = [torch.empty(n, H, d, device="cuda") for _ in range(2)]
        for pool, slots, o in zip((small, big), at, out):
            pool.slots()[slots[0]:slots[-1] + 1] = 0      # (bytes between blocks are no one's)
            pool.pack(slots, S0)
            pool.decay_step(slots, *x, alpha, o)
            assert pool.get_error() == 0
        assert torch.equal(*out)
        assert torch.equal(small.slots(), big.slots()[n_slots - n:])
        small.close(), big.close()
