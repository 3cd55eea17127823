"""States of the bf16 128 x 128 prompt kernels on inputs where 64-token blocks are at their worst: equal,
alternating and few keys with beta |k|^2 up to 2, keys of any length, values that cancel."""
import pytest
import torch

import quantized_linear_attention_damp_b200 as D
from tests.prefill_helpers import EPS32, EPS_BF16, recurrence

pytestmark = pytest.mark.gpu

B = 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# A state may be off by 16 times what the block form in FP32 arithmetic is off by on the same inputs, and by
# 16 half steps of the largest it was.  Half steps of the kernels between two states: operands of products
# T' 3 (A's two factors, the inverse), R 2, diag(w) U 2; sums of up to 24 matrix instructions, truncated (2
# each) and independent: 2 sqrt(24) = 9.8; in all 16, where the FP32 form has one at least.
# A readout is rounded to bf16, and the operands of its products (S in Q S, P and U in P U) are pairs of bf16
# values, which leave 2^-17 of them; with the dropped product of two second terms at most 4 such parts.
STEPS, SPLITS = 16, 4 * 2.0 ** -17


def blocks(rule, q, k, v, alpha, beta, S0, dtype):
    """The block form of one request in `dtype` on the CPU: (its state [H][k][v], what the readouts add up in
    absolute values [L][H][v])."""
    x = [t.detach().cpu().to(dtype).transpose(0, 1) for t in (q, k, v, alpha, beta)]
    S, sums = S0.cpu().to(dtype), []
    for at in range(0, v.shape[0], B):
        Q, K, V, a, be = (t[:, at:at + B] for t in x)
        n = K.shape[1]
        Gam = torch.zeros(*a.shape, n, dtype=dtype)                            # product of alpha over s+1..t
        for t in range(n):
            Gam[:, t, :t] = Gam[:, t - 1, :t] * a[:, t, None] if t else 0.0
            Gam[:, t, t] = 1.0
        gam, w = torch.cumprod(a, 1), Gam[:, -1, :, None]
        P = Gam * (Q @ K.transpose(1, 2))
        U = V
        if rule == "delta":
            A = torch.tril(be[..., None] * Gam * (K @ K.transpose(1, 2)), -1)
            I = torch.eye(n, dtype=dtype).expand_as(A)
            T = torch.linalg.solve_triangular(I + A, I, upper=False) * be[:, None]
            U = T @ (V - gam[..., None] * (K @ S))
        sums.append(gam[..., None] * (Q.abs() @ S.abs()) + P.abs() @ U.abs())
        S = gam[:, -1, None, None] * S + K.transpose(1, 2) @ (w * U)
    return S, torch.cat(sums, 1).transpose(0, 1)


def case(name, L, H, g):
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(r(L, H, 128)), unit(r(L, H, 128)), r(L, H, 128)
    alpha, beta = torch.ones(L, H), torch.sigmoid(r(L, H))
    kind, _, top = name.partition(":")
    if kind == "equal":
        k = k[:1].expand(L, H, 128)
    elif kind == "alternating":
        k = k[:1] * torch.tensor([1.0, -1.0]).repeat(L // 2 + 1)[:L, None, None]
    elif kind == "four":
        k = k[:4].repeat(L // 4 + 1, 1, 1)[:L]
    elif kind == "subspace":
        k = unit(torch.einsum("lhj,jhd->lhd", r(L, H, 4), k[:4]))
    elif kind == "long":
        k = k * 30.0
    elif kind == "short":
        k = k * 0.01
    elif kind == "cancel":                     # values that cancel in pairs, under a slow decay
        k, v = k[:1].expand(L, H, 128), v[:1] * torch.tensor([1.0, -1.0]).repeat(L // 2 + 1)[:L, None, None]
        alpha = 0.999 + 0.001 * torch.rand(L, H, generator=g)
    elif kind == "decayed":
        alpha = torch.sigmoid(r(L, H) + 3)
    k = k.bfloat16()
    if top:                                    # beta |k|^2 (with |k|^2 of the rounded keys)
        beta = float(top) / (k.float() ** 2).sum(-1)
    cu = lambda x: x.cuda()  # noqa: E731
    return dict(q=cu(q.bfloat16()), k=cu(k.contiguous()), v=cu(v.bfloat16()), alpha=cu(alpha), beta=cu(beta))


KEYS = ["decayed", "random", "equal:1", "equal:1.9", "alternating:1.9", "four:1.9", "subspace:1.9", "random:1.9",
        "long:1.9", "short:1.9", "cancel:1", "cancel:0.3"]


@pytest.mark.parametrize("past", [0, 1])
@pytest.mark.parametrize("rule,name", [("delta", n) for n in KEYS] +
                         [("decay", n) for n in ("decayed", "random", "long", "short", "cancel")])
def test_states_are_as_good_as_fp32_sums(rule, name, past):
    H, lengths = 3, [512, 100, 64]
    g = torch.Generator().manual_seed(sum(map(ord, name)) + past)
    T = sum(lengths)
    x = case(name, T, H, g)
    pool = D.DampPool("fp32", 3, H, 128)
    S0 = (torch.randn(3, H, 128, 128, generator=g) * past).cuda()
    pool.pack(i32([0, 1, 2]), S0)
    plan = D.BatchPlan(3, T, 3).build(i32(lengths), i32([2, 0, 1]), i32([past] * 3))
    out = pool.prefill(plan, x["q"], x["k"], x["v"], x["alpha"], x["beta"] if rule == "delta" else None, rule=rule)
    S1 = torch.empty_like(S0)
    pool.unpack(i32([0, 1, 2]), S1)
    assert pool.get_error() == 0
    pool.close()
    at, worst = 0, []
    for r, L in enumerate(lengths):
        y = [x[c][at:at + L] for c in ("q", "k", "v", "alpha", "beta")]
        slot = [2, 0, 1][r]
        o, S, top = recurrence(rule, *y, S0[slot])
        norm = lambda e: e.double().flatten(1).norm(dim=1)  # noqa: E731
        plain = norm(blocks(rule, *y, S0[slot], torch.float32)[0].cuda() - S)
        lim = STEPS * (plain + EPS32 * top)
        worst.append((norm(S1[slot] - S) / lim).max().item())
        sums = blocks(rule, *y, S0[slot], torch.float64)[1].cuda()
        room = SPLITS * sums + (lim[None] * y[0].double().norm(dim=-1))[..., None]     # (q reads the state's error)
        assert ((out[at:at + L].double() - o).abs() <= EPS_BF16 * o.abs() + room).all()
        at += L
    assert max(worst) <= 1.0, worst


@pytest.mark.parametrize("rule", ["decay", "delta"])
@pytest.mark.parametrize("L,H", [(64, 32), (4096, 32), (4000, 100), (9000, 3)])
def test_constant_decays_over_long_prompts(rule, L, H):
    """Without keys a state is its first one times the product of all decays.  A head's decay is the same for every
    token, so every block's product is off by the same amount: one rounding of it and one of the state's update a
    block are what FP32 allows.  (Few heads: the decay rule cuts the request into segments.)"""
    g = torch.Generator().manual_seed(L)
    a = 1 - 0.5 ** (8 + 6 * torch.rand(H, generator=g, dtype=torch.float64))
    a = a.float()
    S0 = torch.randn(1, H, 128, 128, generator=g).cuda()
    zero = torch.zeros(L, H, 128, dtype=torch.bfloat16, device="cuda")
    v, beta = torch.ones_like(zero), torch.ones(L, H, device="cuda")
    pool = D.DampPool("fp32", 1, H, 128)
    pool.pack(i32([0]), S0)
    plan = D.BatchPlan(1, L, 1).build(i32([L]), i32([0]), i32([1]))
    pool.prefill(plan, zero, zero, v, a.expand(L, H).contiguous().cuda(), beta if rule == "delta" else None, rule=rule)
    S1 = torch.empty_like(S0)
    pool.unpack(i32([0]), S1)
    assert pool.get_error() == 0
    pool.close()
    want = (a.double() ** L).cuda()[:, None, None] * S0[0].double()
    err = (S1[0].double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert (err <= 2 * -(-L // B) * EPS32).all(), err.max()
