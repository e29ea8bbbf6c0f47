"""The gated linear recurrence (prefill, decode step, backward) and the state remap, as cases to measure.

The recurrence, per (batch, key/value head) with a log decay g_t, and its readout per query head:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T          (64 x 64, g_t = -inf starts from nothing)
    y_t = scale * S_t^T q_t

The remap moves the slots of a pool of states: new[i] = old[map[i]], zeros where map[i] is -1.

`run` computes them in elementary torch operations, or, where `own` is true, by the calls a user makes.
"""
import math

import torch

own = False

D = 64                 # head size of keys and values
C = 64                 # tokens of a chunk in the plain forms
SCALE = 0.125          # 1 / sqrt(64)
PACKED_ROWS = 2145     # rows of one packed prefix state of the quadratic kernel, 65 fp32 values each


def listed():
    return [
        # a batch of long prompts of a model with 32 query and 8 key/value heads: the largest forward pass
        dict(name="prefill_batch_8192", op="prefill", dtype="bf16", B=4, Hq=32, Hkv=8, T=8192, ragged=False, cut=0.0, cont=False),
        # one very long prompt, 14 query and 2 key/value heads, with documents packed into it
        dict(name="prefill_long_65536", op="prefill", dtype="bf16", B=1, Hq=14, Hkv=2, T=65536, ragged=False, cut=0.0005, cont=False),
        # the next turn of 64 chats: short prompts of unequal lengths on top of their states
        dict(name="prefill_turns_201", op="prefill", dtype="bf16", B=64, Hq=14, Hkv=2, T=201, ragged=True, cut=0.0, cont=True),
        # fp32 checks and calibration runs, an odd length
        dict(name="prefill_fp32_777", op="prefill", dtype="f32", B=2, Hq=4, Hkv=4, T=777, ragged=False, cut=0.002, cont=False),
        # one chat's next token
        dict(name="decode_one", op="decode", dtype="bf16", B=1, Hq=14, Hkv=2, spare=0),
        # a serving batch of 64 whose states sit in a larger pool
        dict(name="decode_batch_64", op="decode", dtype="bf16", B=64, Hq=32, Hkv=8, spare=16),
        # a large fp32 batch, heads not shared, an odd number of sequences
        dict(name="decode_fp32_301", op="decode", dtype="f32", B=301, Hq=8, Hkv=8, spare=3),
        # a training step of the layer on 4 sequences
        dict(name="backward_batch_4096", op="backward", dtype="bf16", B=4, Hq=32, Hkv=8, T=4096, ragged=False, cut=0.0, cont=False),
        # a training step on packed documents that goes on from a state and passes its gradient back
        dict(name="backward_packed_8191", op="backward", dtype="bf16", B=1, Hq=14, Hkv=2, T=8191, ragged=False, cut=0.002, cont=True),
        # an fp32 gradient check of two padded sequences
        dict(name="backward_fp32_513", op="backward", dtype="f32", B=2, Hq=4, Hkv=2, T=513, ragged=True, cut=0.0, cont=True),
        # beam search: 64 beams take over their parents' packed prefix states (2 heads)
        dict(name="remap_beams_64", op="remap", n=64, floats=2 * PACKED_ROWS * 65, kind="beams"),
        # a pool of 1024 gated states (8 heads): finished sequences are freed, the others move together
        dict(name="remap_compact_1024", op="remap", n=1024, floats=8 * D * D, kind="compact"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "backward", "backward", "remap"])
    if op == "remap":
        floats = rng.choice([1, 2, 4, 8]) * rng.choice([D * D, PACKED_ROWS * 65 // 4 * 4])
        n = _log_int(rng, 2, min(2048, (1 << 25) // floats))
        return dict(op=op, n=n, floats=floats, kind=rng.choice(["beams", "compact"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    rho = rng.choice([1, 2, 4, 5, 7])
    if op == "decode":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 400), Hq=Hkv * rho, Hkv=Hkv, spare=rng.choice([0, 0, 1, 17]))
    most = (1 << 20) if op == "prefill" else (1 << 18)     # tokens x query heads
    if dtype == "f32":
        most >>= 4
    T = _log_int(rng, 1, 65536 if op == "prefill" else 8192)
    T = max(1, min(T, most // (Hkv * rho)))
    B = _log_int(rng, 1, max(1, min(64, most // (Hkv * rho * T))))
    return dict(op=op, dtype=dtype, B=B, Hq=Hkv * rho, Hkv=Hkv, T=T, ragged=rng.random() < 0.4,
                cut=rng.choice([0.0, 0.0, 0.003, 0.03]), cont=rng.random() < 0.5)


def _maps(case, seed):
    """The remap's table: which old slot each new slot takes (-1: none)."""
    gen = torch.Generator().manual_seed(seed + 17)
    n = case["n"]
    if case["kind"] == "beams":        # every slot takes a parent's state; some parents take several
        m = torch.randint(0, n, (n,), generator=gen)
    else:                              # half of the slots live on, moved together; the rest are freed
        live = (torch.rand(n, generator=gen) < 0.5).nonzero().flatten()
        m = torch.full((n,), -1, dtype=torch.int64)
        m[: live.numel()] = live
    return m.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    f32 = torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=f32)

    if case["op"] == "remap":
        m = _maps(case, seed)
        rows = (m != torch.arange(case["n"], dtype=torch.int32)).nonzero().flatten()
        return dict(case=case, pool=normal(case["n"], case["floats"]), map=m.to(dev), rows=rows.to(dev), source=m[rows].long().to(dev))

    dt = torch.bfloat16 if case["dtype"] == "bf16" else f32
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    # heads forget over about 2 to 2000 tokens, as trained gates do; g = log(sigmoid(logit))
    span = torch.logspace(0.3, 3.3, Hkv, device=dev) if Hkv > 1 else torch.full((1,), 200.0, device=dev)
    bias = torch.log(span)

    def gates(*tail):
        logit = normal(B, Hkv, *tail) + bias.view(1, Hkv, *[1] * len(tail))
        return torch.nn.functional.logsigmoid(logit)

    if case["op"] == "decode":
        n = B + case["spare"]
        slots = torch.randperm(n, generator=torch.Generator().manual_seed(seed + 3))[:B].to(torch.int32).to(dev)
        return dict(case=case, q=normal(B, Hq, D).to(dt), k=normal(B, Hkv, D).to(dt), v=normal(B, Hkv, D).to(dt), g=gates(),
                    state=normal(n, Hkv, D, D), slots=slots)

    T = case["T"]
    s = dict(case=case, Q=normal(B, Hq, T, D).to(dt), K=normal(B, Hkv, T, D).to(dt), V=normal(B, Hkv, T, D).to(dt), g=gates(T), lengths=None)
    if case["cut"]:
        first = torch.rand(B, Hkv, T, generator=gen, device=dev)[:, :1]    # a document starts for all heads at once
        s["g"] = torch.where(first < case["cut"], -math.inf, s["g"]).contiguous()
    if case["ragged"]:
        s["lengths"] = torch.randint(T // 4, T + 1, (B,), generator=torch.Generator().manual_seed(seed + 5)).to(torch.int32).to(dev)
    if case["op"] == "prefill":
        s["state"] = normal(B, Hkv, D, D) if case["cont"] else torch.zeros(B, Hkv, D, D, device=dev)
        s["Y"] = torch.zeros(B, Hq, T, D, device=dev, dtype=dt)
        return s
    s["dY"] = normal(B, Hq, T, D).to(dt)
    s["state0"] = normal(B, Hkv, D, D) if case["cont"] else None
    s["dstate"] = normal(B, Hkv, D, D) if case["cont"] else None
    for name in ("Q", "K", "V", "g"):
        s["d" + name] = torch.zeros_like(s[name])
    return s


# ------------------------------------------------------------------ plain forms

def _split(x, N):
    """[B, H, T, ...] -> [B, H, N, C, ...], zeros behind T."""
    B, H, T = x.shape[:3]
    pad = N * C - T
    if pad:
        x = torch.cat([x, x.new_zeros(B, H, pad, *x.shape[3:])], 2)
    return x.reshape(B, H, N, C, *x.shape[3:])


def _live(s, T):
    t = torch.arange(T, device=s["K"].device)
    return t.view(1, T) < s["lengths"].view(-1, 1) if s["lengths"] is not None else t.view(1, T) >= 0


def _decays(s, live, N):
    """Per chunk: `pair` exp(G_i - G_j) for j <= i, `head` exp(G_i) from the chunk's start, `tail` from behind a
    token to its end; `across` [n, m] from the end of chunk m to the start of chunk n, `first` from token 0 to the
    start of chunk n, `last` from the end of chunk m to the end.  Sums of logs in 64 bits, resets counted apart."""
    g = torch.where(live[:, None], s["g"], torch.zeros((), device=s["g"].device))
    g = _split(g, N)
    cut = g == -math.inf
    G = torch.where(cut, torch.zeros_like(g), g).double().cumsum(-1)
    R = cut.long().cumsum(-1)
    no = torch.full((), -math.inf, device=g.device)
    order = torch.arange(C, device=g.device)
    x = (G[..., :, None] - G[..., None, :]).float()
    pair = torch.where((R[..., :, None] == R[..., None, :]) & (order[:, None] >= order), x, no).exp()
    head = torch.where(R == 0, G.float(), no).exp()
    tail = torch.where(R == R[..., -1:], (G[..., -1:] - G).float(), no).exp()
    ends, cuts = G[..., -1].cumsum(-1), R[..., -1].cumsum(-1)      # from token 0 to the end of each chunk
    starts, before = ends - G[..., -1], cuts - R[..., -1]
    n = torch.arange(N, device=g.device)
    x = (starts[..., :, None] - ends[..., None, :]).float()
    across = torch.where((before[..., :, None] == cuts[..., None, :]) & (n[:, None] > n), x, no).exp()
    first = torch.where(before == 0, starts.float(), no).exp()
    last = torch.where(cuts == cuts[..., -1:], (ends[..., -1:] - ends).float(), no).exp()
    return pair, head, tail, across, first, last


def _mix(weights, states):
    """[B,H,N,M] x [B,H,M,D,D] -> [B,H,N,D,D]"""
    return (weights @ states.flatten(-2)).unflatten(-1, (D, D))


def _heads(x, Hkv, N):
    """[B, Hq, T, D] -> [B, Hkv, rho, N, C, D] in 32 bits"""
    return _split(x.float(), N).unflatten(1, (Hkv, x.shape[1] // Hkv))


def _keys(s, live, N):
    zero = torch.zeros((), device=s["K"].device)
    return tuple(_split(torch.where(live[:, None, :, None], s[x].float(), zero), N) for x in ("K", "V"))


def _rows(x, like, live):
    """[B, ..., N, C, ...] back to the layout of `like`; rows that are not live stay as they are in `like`."""
    B, H, T = like.shape[:3]
    x = x.reshape(B, H, -1, *like.shape[3:])[:, :, :T]
    return torch.where(live.view(live.shape[0], 1, T, *[1] * (like.dim() - 3)), x.to(like.dtype), like)


def _plain_prefill(s):
    T, Hkv = s["K"].shape[2], s["K"].shape[1]
    N = -(-T // C)
    live = _live(s, T)
    pair, head, tail, across, first, last = _decays(s, live, N)
    K, V = _keys(s, live, N)
    Q = _heads(s["Q"], Hkv, N)
    chunk = (K * tail[..., None]).transpose(-1, -2) @ V
    before = _mix(across, chunk)
    after = _mix(last[..., None, :], chunk)[:, :, 0]
    if s["case"]["cont"]:
        before = before + first[..., None, None] * s["state"][:, :, None]
        after = after + (first[..., -1] * head[..., -1, -1])[..., None, None] * s["state"]
    y = (Q @ K[:, :, None].transpose(-1, -2) * pair[:, :, None]) @ V[:, :, None]
    y = SCALE * (y + head[:, :, None, ..., None] * (Q @ before[:, :, None]))
    s["Y"].copy_(_rows(y, s["Y"], live))
    s["state"].copy_(after)
    return s["Y"], s["state"]


def _plain_decode(s):
    at = s["slots"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, Hkv = k.shape[:2]
    S = s["state"][at] * s["g"].exp()[..., None, None] + k[..., :, None] * v[..., None, :]
    y = SCALE * (q.view(B, Hkv, -1, D) @ S)
    s["state"][at] = S
    return y.view(B, -1, D).to(s["q"].dtype), s["state"]


def _plain_backward(s):
    T, Hkv = s["K"].shape[2], s["K"].shape[1]
    N = -(-T // C)
    live = _live(s, T)
    pair, head, tail, across, first, last = _decays(s, live, N)
    K, V = _keys(s, live, N)
    zero = torch.zeros((), device=K.device)
    Q, dY = (_heads(torch.where(live[:, None, :, None], s[x].float(), zero), Hkv, N) for x in ("Q", "dY"))
    head_q = head[:, :, None, ..., None]
    whole = head[..., -1]                                          # decay over each chunk
    chunk = (K * tail[..., None]).transpose(-1, -2) @ V
    before = _mix(across, chunk)                                   # state at each chunk's start
    read = SCALE * ((Q * head_q).transpose(-1, -2) @ dY).sum(2)    # its gradient from the chunk's own rows
    end = _mix(across.transpose(-1, -2), read)                     # gradient of the state at each chunk's end
    if s["state0"] is not None:
        before = before + first[..., None, None] * s["state0"][:, :, None]
    if s["dstate"] is not None:
        end = end + last[..., None, None] * s["dstate"][:, :, None]
    Kr, Vr = K[:, :, None], V[:, :, None]
    qk = Q @ Kr.transpose(-1, -2) * pair[:, :, None]
    dp = SCALE * (dY @ Vr.transpose(-1, -2))
    z = dp * pair[:, :, None]
    q_far = SCALE * head_q * (dY @ before[:, :, None].transpose(-1, -2))
    k_far = tail[..., None] * (V @ end.transpose(-1, -2))
    dQ = z @ Kr + q_far
    dK = (z.transpose(-1, -2) @ Q).sum(2) + k_far
    dV = SCALE * (qk.transpose(-1, -2) @ dY).sum(2) + tail[..., None] * (K @ end)
    # a log decay at t lies on every path from j < t to l >= t, inside the chunk or past its ends
    w = torch.tril((qk * dp).sum(2), -1).double()
    rows = w.sum(-1) - w.sum(-2) + (Q * q_far).sum(-1).sum(2).double()
    far = (K * k_far).sum(-1).double()
    dg = rows.flip(-1).cumsum(-1).flip(-1) + far.cumsum(-1) - far
    dg = (dg + (whole * (before * end).sum((-1, -2)))[..., None].double()).float()
    dg = torch.where(_split(s["g"], N) == -math.inf, zero, dg)
    out = [_rows(x, s[n], live) for x, n in ((dQ, "dQ"), (dK, "dK"), (dV, "dV"), (dg, "dg"))]
    for name, x in zip(("dQ", "dK", "dV", "dg"), out):
        s[name].copy_(x)
    if s["state0"] is None:
        return s["dQ"], s["dK"], s["dV"], s["dg"]
    return s["dQ"], s["dK"], s["dV"], s["dg"], read[:, :, 0] + whole[:, :, 0, None, None] * end[:, :, 0]


def _plain_remap(s):
    source = s["source"]
    moved = torch.where((source >= 0)[:, None], s["pool"][source.clamp(min=0)], torch.zeros((), device=source.device))
    s["pool"][s["rows"]] = moved
    return s["pool"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "decode": _plain_decode, "backward": _plain_backward, "remap": _plain_remap}[op](s)
    from grouped_quadratic_gb300 import oal
    if op == "prefill":
        return oal.oal_gated_prefill(s["Q"], s["K"], s["V"], s["g"], SCALE, lengths=s["lengths"], state=s["state"],
                                     continue_from_state=s["case"]["cont"], Y=s["Y"])
    if op == "decode":
        y = oal.oal_gated_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], SCALE, slots=s["slots"])
        return y, s["state"]
    if op == "backward":
        out = oal.oal_gated_backward(s["Q"], s["K"], s["V"], s["g"], s["dY"], SCALE, lengths=s["lengths"], state0=s["state0"],
                                     dstate=s["dstate"], dQ=s["dQ"], dK=s["dK"], dV=s["dV"], dg=s["dg"])
        return out if s["state0"] is not None else out[:4]
    return oal.oal_state_remap(s["pool"], s["map"])


# ------------------------------------------------------------------ work and exact values

def work(case):
    op = case["op"]
    if op == "remap":
        # expected over the tables: a beam's parent is read once however many take it; a freed slot is written only
        n, slot = case["n"], 4 * case["floats"]
        if case["kind"] == "beams":
            return {"bytes": int(slot * n * (1.0 + 1.0 - math.exp(-1.0))), "flops": 0}
        return {"bytes": int(slot * (n / 2 + n)), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    if op == "decode":
        return {"bytes": B * (Hkv * D * D * 8 + e * D * (2 * Hq + 2 * Hkv) + 4 * Hkv), "flops": B * D * D * (3 * Hkv + 2 * Hq)}
    T = case["T"] * (0.625 if case["ragged"] else 1.0)
    states = B * Hkv * D * D * 4
    # the recurrence itself, token by token: update 3 D^2 a key/value head, readout 2 D^2 a query head
    if op == "prefill":
        return {"bytes": int(B * T * (e * D * (2 * Hq + 2 * Hkv) + 4 * Hkv)) + states * (2 if case["cont"] else 1),
                "flops": int(B * T * D * D * (3 * Hkv + 2 * Hq))}
    return {"bytes": int(B * T * (e * D * (3 * Hq + 4 * Hkv) + 8 * Hkv)) + states * (3 if case["cont"] else 0),
            "flops": int(B * T * D * D * (12 * Hkv + 4 * Hq))}


def exact(case, seed):
    """The definitions in 64 bits, one token after another."""
    s = prepare(case, seed)
    if case["op"] == "remap":
        new = s["pool"].double()
        for i, j in enumerate(s["map"].tolist()):
            new[i] = s["pool"][j].double() if j >= 0 else 0.0
        return new
    if case["op"] == "decode":
        pool = s["state"].double()
        ys = []
        for b, at in enumerate(s["slots"].tolist()):
            S = pool[at]
            S.mul_(s["g"][b].double().exp().view(-1, 1, 1)).add_(torch.einsum("hd,he->hde", s["k"][b].double(), s["v"][b].double()))
            q = s["q"][b].double().view(S.shape[0], -1, D)
            ys.append(SCALE * torch.einsum("hrd,hde->hre", q, S).reshape(-1, D))
        return torch.stack(ys), pool

    B, Hq, Hkv, T = case["B"], case["Hq"], case["Hkv"], case["T"]
    if T > 70000 or B * Hq * T > 1 << 21:
        return None
    rho = Hq // Hkv
    n = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    on = torch.tensor([[t < x for x in n] for t in range(T)], device="cuda")
    always = min(n)
    a = s["g"].double().exp()
    k, v = s["K"].double(), s["V"].double()
    q = s["Q"].double().view(B, Hkv, rho, T, D)
    start = s.get("state") if case["op"] == "prefill" else s["state0"]
    S = start.double().clone() if case["cont"] else torch.zeros(B, Hkv, D, D, dtype=torch.float64, device="cuda")
    back = case["op"] == "backward"
    dy = s["dY"].double().view(B, Hkv, rho, T, D) if back else None
    rows = torch.zeros(B, Hkv, rho, T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        new = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        S = new if t < always else torch.where(on[t].view(B, 1, 1, 1), new, S)
        if back:
            rows[:, :, :, t] = SCALE * (dy[:, :, :, t] @ S.transpose(-1, -2))
        else:
            rows[:, :, :, t] = SCALE * (q[:, :, :, t] @ S)
    mask = on.t().view(B, 1, T, 1)
    if not back:
        return torch.where(mask, rows.view(B, Hq, T, D), 0.0), S
    R = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(S)
    ends = (R * S).sum((-1, -2))
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(T)):
        new = R + SCALE * (q[:, :, :, t].transpose(-1, -2) @ dy[:, :, :, t])
        R = new if t < always else torch.where(on[t].view(B, 1, 1, 1), new, R)
        dk[:, :, t] = (R @ v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (R.transpose(-1, -2) @ k[:, :, t, :, None])[..., 0]
        new = a[:, :, t, None, None] * R
        R = new if t < always else torch.where(on[t].view(B, 1, 1, 1), new, R)
    rows, dk, dv = rows * mask.unsqueeze(2), dk * mask, dv * mask
    # d/dg_t = exp(g_t) <S_{t-1}, dS_t>: the sum over l >= t of q_l . dq_l - k_l . dk_l, and <S_T, dS_T>
    x = (q * rows).sum(-1).sum(2) - (k * dk).sum(-1)
    dg = (x.flip(-1).cumsum(-1).flip(-1) + ends[..., None]) * mask[..., 0]
    dg = torch.where(s["g"] == -math.inf, 0.0, dg)
    out = (rows.view(B, Hq, T, D), dk, dv, dg)
    return out + (R,) if s["state0"] is not None else out
