"""The operators around the decode step: request plans, the decay-rule step and prompt prefill.

``run`` computes them in plain torch form, or, where ``own`` is true, through the calls a user makes
(``BatchPlan.build``, ``DampPool.decay_step``, ``DampPool.prefill``).

Cases are dicts with an "op":

* "plan": request lengths -> row offsets, slot maps and the 64-token block table of a ragged batch.
* "step": one token of a decayed linear-attention layer on a pool of recurrent states.
* "prefill": prompts of a ragged batch through a decayed ("decay") or gated delta rule ("delta")
  layer, states read from and left in an FP32 pool.
"""
import math

import torch

own = False

BLOCK = 64


def listed():
    return [
        # a small serving step's batch: mostly decodes, some prompt pieces
        dict(name="plan_16", op="plan", n=16, tokens=512, past=True),
        # a whole cluster queue planned at once: 4096 requests, a million prompt tokens
        dict(name="plan_4096", op="plan", n=4096, tokens=1 << 20, past=True),
        # two users decoding: the latency of one layer's step on the mixed FP16/INT8 pool
        dict(name="step_mixed_2x32", op="step", n=2, H=32, Hqk=32, dk=128, dv=128, fmt="mixed",
             hp=27, dtype="bf16"),
        # FP32 inputs, a state that is not square, q/k heads shared by two value heads, INT8 pool
        dict(name="step_int8_48x8_96x160", op="step", n=48, H=8, Hqk=4, dk=96, dv=160, fmt="int8",
             hp=0, dtype="f32"),
        # the high-concurrency batch on FP32 states: pure HBM bandwidth
        dict(name="step_fp32_512x48", op="step", n=512, H=48, Hqk=48, dk=128, dv=128, fmt="fp32",
             hp=0, dtype="bf16"),
        # a handful of short user turns
        dict(name="decay_short", op="prefill", rule="decay", n=8, tokens=200, H=32, Hqk=32, dk=128,
             dv=128, dtype="bf16", past=False, pad=0),
        # a prefill batch of ragged prompts, half of them continued, one padding entry
        dict(name="decay_ragged", op="prefill", rule="decay", n=16, tokens=8192, H=32, Hqk=16,
             dk=128, dv=128, dtype="bf16", past=True, pad=1),
        # one long prompt: little parallelism over requests
        dict(name="decay_long", op="prefill", rule="decay", n=1, tokens=4096, H=32, Hqk=32, dk=128,
             dv=128, dtype="bf16", past=False, pad=0),
        dict(name="delta_short", op="prefill", rule="delta", n=8, tokens=200, H=32, Hqk=32, dk=128,
             dv=128, dtype="bf16", past=False, pad=0),
        dict(name="delta_long", op="prefill", rule="delta", n=1, tokens=8192, H=32, Hqk=16, dk=128,
             dv=128, dtype="bf16", past=False, pad=0),
        dict(name="delta_ragged", op="prefill", rule="delta", n=16, tokens=16384, H=32, Hqk=32,
             dk=128, dv=128, dtype="bf16", past=True, pad=1),
        # FP32 inputs on the smaller state
        dict(name="delta_f32_64", op="prefill", rule="delta", n=4, tokens=700, H=8, Hqk=8, dk=64,
             dv=64, dtype="f32", past=True, pad=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "step", "step", "prefill", "prefill", "prefill"])
    if op == "plan":
        n = _log_int(rng, 1, 4096)
        return dict(op="plan", n=n, tokens=_log_int(rng, n, 1 << 20), past=rng.random() < 0.7)
    if op == "step":
        fmt = rng.choice(["fp32", "mixed", "int8", "fp8"])
        if rng.random() < 0.6:
            dk = dv = 128
        else:
            dk, dv = 16 * rng.randint(1, 16), 16 * rng.randint(1, 16)
        Hqk = rng.choice([1, 2, 4, 8, 16])
        H = Hqk * rng.choice([1, 2, 3])
        top = (512 * 48 * 128 * 128) // (2 * H * dk * dv)
        n = _log_int(rng, 1, max(1, min(512, top)))
        hp = rng.randint(0, dk) if fmt == "mixed" else 0
        return dict(op="step", n=n, H=H, Hqk=Hqk, dk=dk, dv=dv, fmt=fmt, hp=hp,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    rule = rng.choice(["decay", "delta"])
    if rng.random() < 0.7:
        dk = dv = 128
        dtype, most = "bf16", 8192 if rule == "delta" else 4096
    else:
        dk, dv = 16 * rng.randint(1, 16), 16 * rng.randint(1, 16)
        dtype, most = rng.choice(["bf16", "f32"]), 2048
    Hqk = rng.choice([1, 2, 4, 8, 16])
    H = Hqk * rng.choice([1, 2])
    tokens = _log_int(rng, 1, most)
    n = _log_int(rng, 1, min(24, tokens))
    return dict(op="prefill", rule=rule, n=n, tokens=tokens, H=H, Hqk=Hqk, dk=dk, dv=dv,
                dtype=dtype, past=rng.random() < 0.5, pad=1 if n > 3 and rng.random() < 0.5 else 0)


# ------------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _lengths(case, g):
    """n lengths that add up to at most `tokens`, the longest at most ~4 times the mean; with many
    requests one in sixteen is empty."""
    n, tokens = case["n"], case["tokens"]
    w = 0.25 + 0.75 * torch.rand(n, generator=g, dtype=torch.float64)
    if n >= 8:
        w[torch.rand(n, generator=g) < 1 / 16] = 0
    return (w / w.sum().clamp_min(1e-9) * tokens).floor().to(torch.int32)


def _requests(case, seed, device):
    g = _gen(seed * 7 + 1, "cpu")
    n = case["n"]
    length = _lengths(case, g)
    slots = n + 3
    slot = torch.randperm(slots, generator=g)[:n].to(torch.int32)
    pad = case.get("pad", 1 if n >= 8 else 0)
    if pad:
        slot[:pad] = -1
    past = torch.randint(1, 4096, (n,), generator=g, dtype=torch.int32)
    past[torch.rand(n, generator=g) < 0.5] = 0
    if not case["past"]:
        past.zero_()
    return dict(lengths=length.to(device), slot_idx=slot.to(device), past=past.to(device),
                n_slots=slots, longest=int(length.max()))


def _unit(shape, g, dtype):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _alpha(shape, H, g):
    """Fresh decays of heads whose half-lives spread over 1 .. 4096 tokens."""
    half = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(4096.0))
    z = torch.randn(shape, generator=g, device="cuda")
    return torch.exp(-torch.nn.functional.softplus(z) / half)


def _fp16_rows(case, g):
    """Boolean [H][dk]: the FP16 key rows of each head."""
    if case["fmt"] != "mixed":
        return torch.zeros(case["H"], case["dk"], dtype=torch.bool, device="cuda")
    r = torch.rand(case["H"], case["dk"], generator=g, device="cuda").argsort(dim=-1)
    return r < case["hp"]


def prepare(case, seed):
    dev = "cuda"
    if case["op"] == "plan":
        s = dict(case=case, **_requests(case, seed, dev))
        if own:
            import quantized_linear_attention_damp_b200 as D
            s["plan"] = D.BatchPlan(case["n"], case["tokens"], s["n_slots"])
        return s
    g = _gen(seed, dev)
    H, Hqk, dk, dv = case["H"], case["Hqk"], case["dk"], case["dv"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "step":
        n = case["n"]
        slots = n + (n + 3) // 4
        s = dict(case=case, q=_unit((n, Hqk, dk), g, dt), k=_unit((n, Hqk, dk), g, dt),
                 v=torch.randn((n, H, dv), generator=g, device=dev).to(dt),
                 alpha=_alpha((n, H), H, g), rows=_fp16_rows(case, g))
        s["slot_idx"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
        S0 = 0.1 * torch.randn((slots, H, dk, dv), generator=g, device=dev)
        s["out"] = torch.zeros((n, H, dv), device=dev)
        if own:
            import quantized_linear_attention_damp_b200 as D
            fmt = case["fmt"]
            s["pool"] = D.DampPool(fmt, slots, H, dk, d_v=dv,
                                   fp16_map=s["rows"].cpu().numpy() if fmt == "mixed" else None)
            s["pool"].pack(torch.arange(slots, dtype=torch.int32, device=dev), S0)
            if fmt == "fp32":
                s["states"] = s["pool"].slots().view(torch.float32).view(slots, H, dk, dv)
            else:
                s["states"] = torch.empty((n, H, dk, dv), device=dev)
        elif case["fmt"] == "fp32":
            s["S"] = S0
        else:
            s.update(_quantise(S0, s["rows"], case["fmt"]))
        return s
    s = dict(case=case, **_requests(case, seed, dev))
    T = case["tokens"]
    s.update(q=_unit((T, Hqk, dk), g, dt), k=_unit((T, Hqk, dk), g, dt),
             v=torch.randn((T, H, dv), generator=g, device=dev).to(dt), alpha=_alpha((T, H), H, g),
             beta=torch.sigmoid(torch.randn((T, H), generator=g, device=dev)),
             out=torch.zeros((T, H, dv), dtype=dt, device=dev))
    S0 = 0.1 * torch.randn((s["n_slots"], H, dk, dv), generator=g, device=dev)
    if own:
        import quantized_linear_attention_damp_b200 as D
        s["plan"] = D.BatchPlan(case["n"], T, s["n_slots"])
        s["plan"].build(s["lengths"], s["slot_idx"], s["past"])
        s["pool"] = D.DampPool("fp32", s["n_slots"], H, dk, d_v=dv)
        s["pool"].pack(torch.arange(s["n_slots"], dtype=torch.int32, device=dev), S0)
        s["S"] = s["pool"].slots().view(torch.float32).view(s["n_slots"], H, dk, dv)
    else:
        s["S"] = S0
        s["cu"] = torch.nn.functional.pad(s["lengths"].cumsum(0), (1, 0))
    return s


# ------------------------------------------------------------------- plain forms

def _plain_plan(s):
    n, T = s["case"]["n"], s["case"]["tokens"]
    blocks = (T + (BLOCK - 1) * n) // BLOCK
    length, past = s["lengths"].long(), s["past"].long()
    dev = length.device
    ok = (length > 0) & (s["slot_idx"] >= 0) & (s["slot_idx"] < s["n_slots"])
    store = torch.where(ok, s["slot_idx"], -1)
    load = torch.where(past > 0, store, -1)
    cu = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    cu[1:] = length.cumsum(0)
    nb = (length + BLOCK - 1) // BLOCK
    bcu = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    bcu[1:] = nb.cumsum(0)
    # the request of row t: the number of requests that end at or before it
    at = torch.zeros(T + 1, dtype=torch.int64, device=dev).index_add_(0, cu[1:], torch.ones_like(length))
    req = at.cumsum(0)[:T]
    t = torch.arange(T, device=dev)
    live = req < n
    req = req.clamp(max=n - 1)
    token_slot = torch.where(live, store[req], -1)
    token_pos = torch.where(live, past[req] + t - cu[req], -1)
    at = torch.zeros(blocks + 1, dtype=torch.int64, device=dev).index_add_(0, bcu[1:], torch.ones_like(length))
    breq = at.cumsum(0)[:blocks]
    blive = breq < n
    breq = breq.clamp(max=n - 1)
    idx = torch.arange(blocks, device=dev) - bcu[breq]
    table = torch.stack([breq, cu[breq] + idx * BLOCK, (length[breq] - idx * BLOCK).clamp(max=BLOCK),
                         idx], dim=1)
    table = torch.where(blive[:, None], table, -1)
    totals = torch.stack([cu[n], bcu[n], length.max(), torch.zeros_like(cu[n])])
    i32 = torch.int32
    return [cu.to(i32), load.to(i32), store.to(i32), table.to(i32), token_slot.to(i32),
            token_pos.to(i32), totals.to(i32)]


def _row_scale(X, Q):
    """fl(a / Q) and fl(Q / a) of the rows' largest magnitudes a; zeros where a is 0.  Q is a tensor:
    with a Python number torch multiplies by a rounded reciprocal instead of dividing."""
    a = X.abs().amax(dim=-1, keepdim=True)
    Q = torch.full_like(a, Q)
    inv = Q / a
    zero = (a == 0) | torch.isinf(inv)
    return torch.where(zero, 0.0, a / Q), torch.where(zero, 0.0, inv)


def _quantise(X, rows, fmt):
    """The pool formats' stored values of FP32 states X [..][H][dk][dv]."""
    if fmt == "fp8":
        scale, inv = _row_scale(X, 448.0)
        code = (X * inv).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        scale, inv = _row_scale(X, 127.0)
        code = (X.double() * inv.double()).round().to(torch.int8)
    return dict(code=code, scale=scale, half=X.to(torch.float16) if fmt == "mixed" else None)


def _codes(code):
    return code.view(torch.float8_e4m3fn).float() if code.dtype == torch.uint8 else code.float()


def _dequantise(code, scale, half, rows):
    x = _codes(code) * scale
    return x if half is None else torch.where(rows[..., None], half.float(), x)


def _heads(x, H):
    """Shared q/k heads repeated for the H value heads that read them."""
    return x.repeat_interleave(H // x.shape[-2], dim=-2)


def _plain_step(s):
    c = s["case"]
    idx = s["slot_idx"].long()
    q, k = _heads(s["q"].float(), c["H"]), _heads(s["k"].float(), c["H"])
    v = s["v"].float()
    if c["fmt"] == "fp32":
        S = s["S"][idx]
    else:
        half = s["half"]
        S = _dequantise(s["code"][idx], s["scale"][idx], None if half is None else half[idx],
                        s["rows"])
    S = s["alpha"][..., None, None] * S
    # one rounding of k v + S, as a fused multiply-add takes it
    X = (k.double()[..., None] * v.double()[..., None, :] + S).float()
    out = (q[..., None] * X).sum(dim=-2)
    if c["fmt"] == "fp32":
        s["S"][idx] = X
        return [out, s["S"]]
    new = _quantise(X, s["rows"], c["fmt"])
    for name, x in new.items():
        if x is not None:
            s[name][idx] = x
    return [out, _dequantise(new["code"], new["scale"], new["half"], s["rows"])]


def _padded(s, x, fill, L):
    """Rows of the ragged batch as [n][L][...], `fill` behind each request's end."""
    cu = s["cu"]
    t = cu[:-1, None] + torch.arange(L, device=x.device)
    live = t < cu[1:, None]
    y = x[t.clamp(max=x.shape[0] - 1)].float()
    return torch.where(live.view(*live.shape, *([1] * (x.dim() - 1))), y, fill)


def _states_in(s):
    ok = (s["slot_idx"] >= 0) & (s["lengths"] > 0)
    src = torch.where(ok, s["slot_idx"], 0).long()
    load = ok & (s["past"] > 0)
    return ok, src, s["S"][src] * load[:, None, None, None]


def _finish(s, o, S1, ok, src):
    """Rows [n][L][H][dv] and states [n][H][dk][dv] to where the batch keeps them."""
    c, cu = s["case"], s["cu"]
    T, L = c["tokens"], o.shape[1]
    o = torch.where(ok[:, None, None, None], o, 0.0).to(s["v"].dtype)
    t = cu[:-1, None] + torch.arange(L, device=o.device)
    t = torch.where(t < cu[1:, None], t, T)      # row T takes what is behind the ends
    out = torch.cat([s["out"], torch.zeros_like(s["out"][:1])])
    out[t.reshape(-1)] = o.reshape(-1, c["H"], c["dv"])
    S = torch.cat([s["S"], torch.zeros_like(s["S"][:1])])
    S[torch.where(ok, src, s["n_slots"])] = S1
    s["S"].copy_(S[:-1])
    return [out[:T], s["S"]]


def _plain_decay(s):
    """o = (q k^T * decay) v + decay q S0 over each whole request."""
    c, L = s["case"], max(1, s["longest"])
    q = _heads(_padded(s, s["q"], 0.0, L), c["H"]).transpose(1, 2)
    k = _heads(_padded(s, s["k"], 0.0, L), c["H"]).transpose(1, 2)
    v = _padded(s, s["v"], 0.0, L).transpose(1, 2)                     # [n][H][L][dv]
    g = _padded(s, s["alpha"], 1.0, L).transpose(1, 2).double().log().cumsum(-1)
    ok, src, S0 = _states_in(s)
    seen = torch.ones(L, L, dtype=torch.bool, device=q.device).tril()
    P = (g[..., :, None] - g[..., None, :]).masked_fill_(~seen, -math.inf).exp_().float()
    P *= q @ k.transpose(-1, -2)
    o = P @ v + g.exp().float()[..., None] * (q @ S0)
    to_end = (g[..., -1:] - g).exp().float()[..., None]
    S1 = g[..., -1].exp().float()[..., None, None] * S0 + (k * to_end).transpose(-1, -2) @ v
    return _finish(s, o.transpose(1, 2), S1, ok, src)


def _plain_delta(s):
    """Chunks of 64 tokens: (I + A) U = diag(beta)(V - diag(decay) K S), then as the decay rule."""
    c, C = s["case"], BLOCK
    L = max(1, -(-s["longest"] // C)) * C
    n, H, nc = c["n"], c["H"], L // C

    def chunks(x, fill):
        x = _padded(s, x, fill, L)
        x = _heads(x, H) if x.dim() == 4 else x[..., None]
        return x.view(n, nc, C, H, x.shape[-1]).permute(1, 0, 3, 2, 4)   # [nc][n][H][C][.]

    q, k, v = chunks(s["q"], 0.0), chunks(s["k"], 0.0), chunks(s["v"], 0.0)
    beta = chunks(s["beta"], 0.0)
    g = chunks(s["alpha"], 1.0)[..., 0].double().log().cumsum(-1)
    seen = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = (g[..., :, None] - g[..., None, :]).masked_fill(~seen, -math.inf).exp().float()
    kT = k.transpose(-1, -2)
    A = (beta * (k @ kT) * D).tril(-1)
    eye = torch.eye(C, device=q.device)
    inv, power = eye - A, A @ A                # the product of (I + (-A)^(2^i)) is (I + A)^-1
    for _ in range(5):
        inv = inv + inv @ power
        power = power @ power
    P = (q @ kT) * D
    gamma = g.exp().float()[..., None]
    to_end = (g[..., -1:] - g).exp().float()[..., None]
    ok, src, S = _states_in(s)
    outs = []
    for i in range(nc):
        U = inv[i] @ (beta[i] * (v[i] - gamma[i] * (k[i] @ S)))
        outs.append(gamma[i] * (q[i] @ S) + P[i] @ U)
        S = gamma[i][..., -1:, :] * S + kT[i] @ (to_end[i] * U)
    o = torch.stack(outs).permute(1, 0, 3, 2, 4).reshape(n, L, H, c["dv"])
    return _finish(s, o, S, ok, src)


# ------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "plan":
        return _plain_plan(state)
    if op == "step":
        return _plain_step(state)
    return _plain_decay(state) if state["case"]["rule"] == "decay" else _plain_delta(state)


def _own(s, op):
    if op == "plan":
        p = s["plan"]
        p.build(s["lengths"], s["slot_idx"], s["past"])
        return [p.cu_seqlens, p.load_slot, p.store_slot, p.block_table, p.token_slot, p.token_pos,
                p.totals]
    if op == "step":
        s["pool"].decay_step(s["slot_idx"], s["q"], s["k"], s["v"], s["alpha"], s["out"])
        if s["case"]["fmt"] != "fp32":
            s["pool"].unpack(s["slot_idx"], s["states"])
        return [s["out"], s["states"]]
    rule = s["case"]["rule"]
    s["pool"].prefill(s["plan"], s["q"], s["k"], s["v"], s["alpha"],
                      s["beta"] if rule == "delta" else None, s["out"], rule=rule)
    return [s["out"], s["S"]]


def work(case):
    """Bytes and operations one pass cannot do without."""
    n = case["n"]
    if case["op"] == "plan":
        T = case["tokens"]
        blocks = (T + (BLOCK - 1) * n) // BLOCK
        return dict(bytes=12 * n + 4 * (n + 1) + 8 * n + 16 * blocks + 8 * T + 16, flops=n + T)
    H, Hqk, dk, dv = case["H"], case["Hqk"], case["dk"], case["dv"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "step":
        r = dk - case["hp"]
        block = 4 * dk * dv if case["fmt"] == "fp32" else 2 * case["hp"] * dv + r * dv + 4 * r
        read_back = 0 if case["fmt"] == "fp32" else 4 * dk * dv
        rows = n * (2 * Hqk * dk + H * dv) * b + n * H * (4 + 4 * dv) + 4 * n
        return dict(bytes=rows + n * H * (2 * block + read_back), flops=4 * n * H * dk * dv)
    T, delta = case["tokens"], case["rule"] == "delta"
    rows = T * ((2 * Hqk * dk + 2 * H * dv) * b + H * (8 if delta else 4))
    states = n * H * dk * dv * 4 * (1.5 if case["past"] else 1)
    return dict(bytes=rows + states, flops=(6 if delta else 4) * T * H * dk * dv)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """From the recurrences, token by token, in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "plan":
        return None
    H, f8 = case["H"], torch.float64
    rep = lambda x: x.to(f8).repeat_interleave(H // x.shape[-2], dim=-2)  # noqa: E731
    if case["op"] == "step":
        at = s["slot_idx"].long()
        if case["fmt"] == "fp32":
            S = s["S"][at].to(f8)
        else:
            S = _codes(s["code"][at]).to(f8) * s["scale"][at].to(f8)
            if s["half"] is not None:
                S = torch.where(s["rows"][..., None], s["half"][at].to(f8), S)
        S *= s["alpha"].to(f8)[..., None, None]
        S += torch.einsum("nhk,nhv->nhkv", rep(s["k"]), s["v"].to(f8))
        out = torch.einsum("nhk,nhkv->nhv", rep(s["q"]), S)
        if case["fmt"] != "fp32":
            return [out, None]       # which code a value next to a border takes has no 64-bit answer
        full = s["S"].to(f8)
        full[at] = S
        return [out, full]
    cu = [0] + s["lengths"].cumsum(0).tolist()
    slot, past = s["slot_idx"].tolist(), s["past"].tolist()
    length = s["lengths"].tolist()
    n = case["n"]
    out = torch.zeros((case["tokens"], H, case["dv"]), dtype=f8, device="cuda")
    states = s["S"].to(f8)
    go = [r for r in range(n) if length[r] > 0 and slot[r] >= 0]
    go.sort(key=lambda r: -length[r])
    if not go:
        return [out, states]
    dev = "cuda"
    S = torch.stack([states[slot[r]] if past[r] > 0 else torch.zeros_like(states[0]) for r in go])
    start = torch.tensor([cu[r] for r in go], device=dev)
    live = [sum(length[r] > t for r in go) for t in range(length[go[0]])]
    q, k, v = rep(s["q"]), rep(s["k"]), s["v"].to(f8)
    al, be = s["alpha"].to(f8), s["beta"].to(f8)
    for t, m in enumerate(live):
        at = start[:m] + t
        M = S[:m]
        M *= al[at][..., None, None]
        kt, d = k[at], v[at]
        if case["rule"] == "delta":
            d = be[at][..., None] * (d - (kt[..., None, :] @ M)[..., 0, :])
        M += kt[..., None] * d[..., None, :]
        out[at] = (q[at][..., None, :] @ M)[..., 0, :]
    for i, r in enumerate(go):
        states[slot[r]] = S[i]
    return [out, states]
