"""Rotary positions, a paged cache of keys and values and the softmax attention that reads it, as cases to measure.

Rotation of row x at position p (one position an axis; pair r belongs to axis a_r and turns by p[a_r] * freq[r]):

    (x_r, x_{r+32}) -> (x_r cos - x_{r+32} sin, x_{r+32} cos + x_r sin)     halves; pairs: (x_{2r}, x_{2r+1})

and, for gradients, by the opposite angle.  Appending writes the rotated keys and the values of new tokens to the
pages of their sequences and rotates the queries along.  Attention of T new tokens at positions i = past + t over a
sequence's pages, query head h on key/value head h / (Hq / Hkv):

    s_j = scale q.k_j,  s_j = cap tanh(s_j / cap),  s_j = s_j - slope_h |i - j|
    y_i = sum_j softmax(s)_j v_j  over the j that i may see:
          first_i <= j, i - window < j, and j <= i or j < prefix (but inside the sequence)

`run` computes them in elementary torch operations, or, where `own` is true, by the calls a user makes.
"""
import math

import torch

own = False

D = 64                 # head size of keys and values
SCALE = 0.125          # 1 / sqrt(64)
PLAIN = 1 << 28        # scores that the plain form holds at a time


def _attention(name, B, Hq, Hkv, T, past, page, dtype="bf16", ragged=False, cap=0.0, window=0, bias=False, docs=False, prefix=False):
    return dict(name=name, op="attention", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, T=T, past=past, page=page, ragged=ragged, cap=cap,
                window=window, bias=bias, docs=docs, prefix=prefix)


def listed():
    return [
        # a training batch's queries and keys, views of the projection's output, 32 and 8 heads; positions in time,
        # height and width
        dict(name="rope_batch_8192", op="rope", dtype="bf16", B=4, Hq=32, Hkv=8, T=8192, axes=3, form="halves", inverse=False, ragged=False),
        # the gradients of two padded sequences of a check in 32 bits, neighbouring pairs turned
        dict(name="rope_grad_fp32_513", op="rope", dtype="f32", B=2, Hq=4, Hkv=2, T=513, axes=1, form="pairs", inverse=True, ragged=True),
        # a batch of long prompts enters the cache
        dict(name="append_batch_8192", op="append", dtype="bf16", B=4, Hq=32, Hkv=8, T=8192, past=0, page=64, axes=1, form="halves", ragged=False),
        # the next token of a serving batch of 64
        dict(name="append_token_64", op="append", dtype="bf16", B=64, Hq=32, Hkv=8, T=1, past=4096, page=16, axes=1, form="halves", ragged=True),
        # the same batch of long prompts attends: the largest forward pass
        _attention("attend_batch_8192", 4, 32, 8, 8192, 0, 64),
        # the last 2048 tokens of a very long prompt that is read chunk by chunk, 14 query and 2 key/value heads
        _attention("attend_chunk_65536", 1, 14, 2, 2048, 63488, 128),
        # the next turn of 64 chats, unequal lengths; capped scores and a window
        _attention("attend_turns_201", 64, 14, 2, 201, 4096, 16, ragged=True, cap=30.0, window=1024),
        # an image prompt that sees all of itself, then text; documents packed behind one another; distances
        _attention("attend_prefix_1500", 2, 32, 8, 1500, 0, 32, ragged=True, bias=True, docs=True, prefix=True),
        # an fp32 check of an odd length with packed documents
        _attention("attend_fp32_777", 2, 4, 4, 777, 100, 16, dtype="f32", docs=True),
        # one chat's next token
        _attention("attend_token_one", 1, 14, 2, 1, 32768, 64),
        # the next token of a serving batch of 64
        _attention("attend_token_64", 64, 32, 8, 1, 8191, 16, ragged=True),
        # five drafted tokens each for 32 sequences
        _attention("attend_drafts_5", 32, 32, 8, 5, 3000, 32, ragged=True, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7])
    if op != "attention":
        T = 1 if rng.random() < 0.3 else _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(256, (1 << 20) // (Hq * T))))
        case = dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, T=T, axes=rng.choice([1, 1, 3]), form=rng.choice(["halves", "halves", "pairs"]),
                    ragged=rng.random() < 0.4)
        if op == "rope":
            return dict(case, inverse=rng.random() < 0.5)
        past = min(_log_int(rng, 1, 65536), (1 << 19) // (B * Hkv))
        return dict(case, past=past, page=rng.choice([16, 32, 64, 128]))
    T = 1 if rng.random() < 0.35 else _log_int(rng, 1, 8192)
    most = 1 << (31 if dtype == "bf16" else 27)            # scores
    B = _log_int(rng, 1, 64)
    while B > 1 and B * Hq * T * T > most:
        B = (B + 1) // 2
    T = max(1, min(T, math.isqrt(most // (B * Hq))))
    past = min(rng.choice([0, _log_int(rng, 1, 65536)]), (1 << 22) // (B * Hkv), most // (B * Hq * T))
    extra = rng.choice(["none", "none", "none", "cap", "window", "bias", "docs", "prefix", "all"])
    on = lambda x: extra in (x, "all")
    return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, T=T, past=past, page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5,
                cap=rng.choice([5.0, 30.0, 50.0]) if on("cap") else 0.0, window=_log_int(rng, 1, 4096) if on("window") else 0,
                bias=on("bias"), docs=on("docs"), prefix=on("prefix"))


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """The pairs' angles a position, in 64 bits, and their axes: sections of 8, 12 and 12 for time, height and width."""
    base = 1e6 if case["op"] == "append" else 1e4
    freq = base ** (-torch.arange(32, dtype=torch.float64) / 32)
    axes = torch.tensor([0] * 8 + [1] * 12 + [2] * 12) if case["axes"] == 3 else torch.zeros(32, dtype=torch.int64)
    return freq, axes


def _lengths(case, gen):
    """Host numbers, as a scheduler has them: new tokens of each sequence and those in the cache before."""
    B, T, past = case["B"], case["T"], case.get("past", 0)
    if not case["ragged"]:
        return [T] * B, [past] * B
    new = torch.randint(max(1, T // 4), T + 1, (B,), generator=gen).tolist()
    return new, torch.randint(past // 4, past + 1, (B,), generator=gen).tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, Hq, Hkv, T = case["B"], case["Hq"], case["Hkv"], case["T"]
    new, past = _lengths(case, host)
    s = dict(case=case, new=new, before=past, lengths=None)
    if case["ragged"]:
        s["lengths"] = torch.tensor(new, dtype=torch.int32, device=dev)
    s["past"] = torch.tensor(past, dtype=torch.int32, device=dev)

    if case["op"] != "attention":
        # the projection's output, [B, T, heads, 64]: queries, keys and values are views of it
        qkv = torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen, device=dev, dtype=torch.float32).to(dt)
        Q, K, V = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
        freq, axes = _frequencies(case)
        s.update(Q=Q, K=K, V=V, freq=freq.to(dev), axes=axes.to(dev), positions=None)
        if case["axes"] == 3:      # time goes on along a video; height and width inside its frames of 24 x 32 patches
            t = torch.arange(T, device=dev) + s["past"][:, None].long()
            s["positions"] = torch.stack([t // 768, t // 32 % 24, t % 32]).to(torch.int32)
        if own:
            from grouped_quadratic_gb300 import oal
            s["form"] = oal.OAL_ROPE_HALVES if case["form"] == "halves" else oal.OAL_ROPE_PAIRS
            s["plan"] = oal.oal_rope_plan(freq, axes, device=dev)
        s["Yq"] = torch.zeros(B, Hq, T, D, device=dev, dtype=dt)
        if case["op"] == "rope":
            s["Yk"] = torch.zeros(B, Hkv, T, D, device=dev, dtype=dt)
            return s

    # every sequence has pages for all of its tokens, spread over a pool that would hold the longest and some to spare
    P = case["page"]
    most = -(-(case["past"] + T) // P)
    need = [-(-(a + b) // P) for a, b in zip(past, new)]
    n = B * most + 7
    order = torch.randperm(n, generator=host).to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    s["table"] = table.to(dev)
    s["Kp"], s["Vp"] = (torch.randn(n, Hkv, P, D, generator=gen, device=dev, dtype=torch.float32).to(dt) for _ in range(2))
    if case["op"] == "append":
        return s

    s["Q"] = (1.5 * torch.randn(B, Hq, T, D, generator=gen, device=dev, dtype=torch.float32)).to(dt)
    s["Y"] = torch.zeros(B, Hq, T, D, device=dev, dtype=dt)
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq) if case["bias"] else None
    s["first"] = s["prefix"] = None
    if case["docs"]:               # a document starts every 300 tokens or so
        t = torch.arange(T, device=dev) + s["past"][:, None].long()
        start = torch.rand(B, T, generator=gen, device=dev) < 1 / 300
        s["first"] = torch.where(start, t, 0).cummax(1).values.to(torch.int32)
    if case["prefix"]:             # the first third of the new tokens, an image, sees all of itself
        s["prefix"] = torch.tensor([a + b // 3 for a, b in zip(past, new)], dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _angles(s):
    """cos and sin [B, 1, T, 32], the angles in 64 bits."""
    T = s["case"]["T"]
    if s["positions"] is not None:
        p = s["positions"][s["axes"]].permute(1, 2, 0).double()
    else:
        p = (s["past"][:, None].double() + torch.arange(T, device=s["past"].device))[..., None]
    a = p * s["freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, form):
    x = x.float()
    if form == "halves":
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _live(s):
    t = torch.arange(s["case"]["T"], device=s["past"].device)
    return t < s["lengths"][:, None] if s["lengths"] is not None else (t >= 0).expand(s["case"]["B"], -1)


def _plain_rope(s):
    cos, sin = _angles(s)
    if s["case"]["inverse"]:
        sin = -sin
    live = _live(s)[:, None, :, None]
    for x, y in (("Q", "Yq"), ("K", "Yk")):
        s[y].copy_(torch.where(live, _turn(s[x], cos, sin, s["case"]["form"]).to(s[y].dtype), s[y]))
    return s["Yq"], s["Yk"]


def _plain_append(s):
    c = s["case"]
    cos, sin = _angles(s)
    live = _live(s)
    s["Yq"].copy_(torch.where(live[:, None, :, None], _turn(s["Q"], cos, sin, c["form"]).to(s["Yq"].dtype), s["Yq"]))
    k = _turn(s["K"], cos, sin, c["form"]).to(s["Kp"].dtype)
    t = s["past"][:, None].long() + torch.arange(c["T"], device=live.device)
    page = s["table"].long().gather(1, (t // c["page"]).clamp(max=s["table"].shape[1] - 1))
    if s["lengths"] is None:
        page, row, k, v = page.flatten(), (t % c["page"]).flatten(), k.transpose(1, 2).flatten(0, 1), s["V"].transpose(1, 2).flatten(0, 1)
    else:
        page, row, k, v = page[live], (t % c["page"])[live], k.transpose(1, 2)[live], s["V"].transpose(1, 2)[live]
    s["Kp"][page, :, row] = k
    s["Vp"][page, :, row] = v
    return s["Yq"], s["Kp"], s["Vp"]


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, T, P = c["B"], c["Hq"], c["Hkv"], c["T"], c["page"]
    total = [a + b for a, b in zip(s["before"], s["new"])]
    keys = max(total)
    pages = s["table"][:, :-(-keys // P)].long().clamp(min=0)
    K, V = (s[x][pages].float().transpose(1, 2).flatten(2, 3) for x in ("Kp", "Vp"))     # [B, Hkv, keys, 64]
    j = torch.arange(K.shape[2], device=K.device)
    ends = s["past"].long() + (s["lengths"].long() if s["lengths"] is not None else T)
    V = torch.where((j < ends[:, None])[:, None, :, None], V, 0.0)
    step = max(1, PLAIN // (B * Hq * K.shape[2]))
    lowest, far = torch.full((), -math.inf, device=K.device), max(s["before"])
    for t0 in range(0, T, step):
        t1 = min(T, t0 + step)
        n = K.shape[2] if c["prefix"] else min(K.shape[2], far + t1)
        i = (s["past"][:, None].long() + torch.arange(t0, t1, device=K.device))[..., None]    # [B, t, 1]
        jj = j[:n]
        see = jj <= i
        if s["prefix"] is not None:
            see = see | (jj < s["prefix"].long()[:, None, None])
        see = see & (jj < ends[:, None, None])
        if c["window"]:
            see = see & (jj > i - c["window"])
        if s["first"] is not None:
            see = see & (jj >= s["first"][:, t0:t1, None])
        q = s["Q"][:, :, t0:t1].float().unflatten(1, (Hkv, Hq // Hkv)).flatten(2, 3)          # [B, Hkv, rho t, 64]
        x = (SCALE * (q @ K[:, :, :n].transpose(-1, -2))).view(B, Hkv, Hq // Hkv, t1 - t0, n)
        if c["cap"]:
            x = c["cap"] * (x / c["cap"]).tanh()
        if s["slopes"] is not None:
            x = x - s["slopes"].view(1, Hkv, -1, 1, 1) * (i - jj).abs().float()[:, None, None]
        x = torch.where(see[:, None, None], x, lowest)
        top = x.amax(-1, keepdim=True)
        x = (x - torch.where(top == -math.inf, 0.0, top)).exp()
        x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
        y = (x.flatten(2, 3) @ V[:, :, :n]).view(B, Hq, t1 - t0, D)
        if s["lengths"] is None:
            s["Y"][:, :, t0:t1] = y.to(s["Y"].dtype)
        else:
            live = (torch.arange(t0, t1, device=K.device) < s["lengths"][:, None])[:, None, :, None]
            s["Y"][:, :, t0:t1] = torch.where(live, y.to(s["Y"].dtype), s["Y"][:, :, t0:t1])
    return s["Y"]


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention}[c["op"]](s)
    from grouped_quadratic_gb300 import oal
    if c["op"] == "rope":
        return oal.oal_rope(s["Q"], s["K"], s["plan"], positions=s["positions"], past=s["past"], lengths=s["lengths"], form=s["form"],
                            inverse=c["inverse"], Yq=s["Yq"], Yk=s["Yk"])
    if c["op"] == "append":
        y = oal.oal_page_append(s["Q"], s["K"], s["V"], s["plan"], s["Kp"], s["Vp"], s["table"], s["past"], positions=s["positions"],
                                lengths=s["lengths"], form=s["form"], Yq=s["Yq"])
        return y, s["Kp"], s["Vp"]
    return oal.oal_paged_attention(s["Q"], s["Kp"], s["Vp"], s["table"], s["past"], lengths=s["lengths"], scale=SCALE, cap=c["cap"],
                                   window=c["window"], slopes=s["slopes"], prefix=s["prefix"], first=s["first"], Y=s["Y"])


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    B, Hq, Hkv, T = c["B"], c["Hq"], c["Hkv"], c["T"]
    rows = B * (T if not c["ragged"] else (max(1, T // 4) + T) / 2)
    if c["op"] == "rope":
        return {"bytes": int(rows * (Hq + Hkv) * D * 2 * e), "flops": int(rows * (Hq + Hkv) * D * 3)}
    if c["op"] == "append":
        return {"bytes": int(rows * (Hq + 2 * Hkv) * D * 2 * e), "flops": int(rows * (Hq + Hkv) * D * 3)}
    # keys that a row sees, and keys that some row of a sequence sees, from expected lengths
    t = rows / B
    past = c["past"] if not c["ragged"] else 0.625 * c["past"]
    sees = past + (t + 1) / 2 + (t / 18 if c["prefix"] else 0)         # the image's tokens see t/6 more on average
    read = past + t
    if c["docs"]:       # a row sees back to its document's start, 300 tokens on average unless the sequence starts later
        p = 1 / 300
        never = (1 - (1 - p) ** t) / (p * t)                            # rows that no document starts before
        sees = min(sees, (past + t / 2) * never + 300 * (1 - never)) if past else min(sees, 300.0)
    if c["window"]:
        sees, read = min(sees, c["window"]), min(read, c["window"] + t)
    return {"bytes": int(B * (2 * t * Hq + 2 * read * Hkv) * D * e), "flops": int(B * Hq * t * sees * 4 * D)}


def _exact_rotation(x, p, s):
    """x [heads, T, 64] in 64 bits, positions p [32, T]: as products of complex numbers."""
    angle = (p.double() * s["freq"][:, None]).T
    if s["case"].get("inverse"):
        angle = -angle
    turn = torch.polar(torch.ones_like(angle), angle)
    x = x.double()
    if s["case"]["form"] == "halves":
        z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous()) * turn).flatten(-2)


def exact(case, seed):
    """The definitions in 64 bits, one sequence after another."""
    s = prepare(case, seed)
    B, Hq, Hkv, T = case["B"], case["Hq"], case["Hkv"], case["T"]
    dev = s["past"].device
    if case["op"] != "attention":
        yq = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=dev)
        yk = torch.zeros(B, Hkv, T, D, dtype=torch.float64, device=dev)
        pools = [s["Kp"].double(), s["Vp"].double()] if case["op"] == "append" else None
        table = s["table"].tolist() if pools else None
        for b, (n, past) in enumerate(zip(s["new"], s["before"])):
            at = torch.arange(past, past + n, device=dev)
            p = s["positions"][s["axes"], b, :n] if s["positions"] is not None else at.expand(32, -1)
            yq[b, :, :n] = _exact_rotation(s["Q"][b, :, :n], p, s)
            yk[b, :, :n] = _exact_rotation(s["K"][b, :, :n], p, s)
            if pools:
                P = case["page"]
                for i in range(past // P, -(-(past + n) // P)):        # page by page
                    lo, hi = max(past, i * P), min(past + n, (i + 1) * P)
                    for pool, rows in zip(pools, (yk[b], s["V"][b].double())):
                        pool[table[b][i], :, lo - i * P:hi - i * P] = rows[:, lo - past:hi - past]
        return (yq, *pools) if pools else (yq, yk)

    if B * Hq * T * (case["past"] + T) > 1 << 34:
        return None
    out = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=dev)
    P, rho = case["page"], Hq // Hkv
    for b, (n, past) in enumerate(zip(s["new"], s["before"])):
        end = past + n
        pages = s["table"][b, :-(-end // P)].long()
        prefix = int(s["prefix"][b]) if s["prefix"] is not None else 0
        for kv in range(Hkv):
            k, v = (s[x][pages, kv].reshape(-1, D)[:end].double() for x in ("Kp", "Vp"))
            block = max(1, (1 << 26) // (rho * end))
            for t0 in range(0, n, block):
                t1 = min(n, t0 + block)
                i = torch.arange(past + t0, past + t1, device=dev)
                hi = torch.maximum(i + 1, torch.full_like(i, prefix)).clamp(max=end)
                lo = torch.zeros_like(i)
                if case["window"]:
                    lo = torch.maximum(lo, i + 1 - case["window"])
                if s["first"] is not None:
                    lo = torch.maximum(lo, s["first"][b, t0:t1].long())
                a, z = int(lo.min()), int(hi.max())
                j = torch.arange(a, z, device=dev)
                x = SCALE * torch.einsum("htd,jd->htj", s["Q"][b, kv * rho:(kv + 1) * rho, t0:t1].double(), k[a:z])
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if s["slopes"] is not None:
                    x -= s["slopes"][kv * rho:(kv + 1) * rho].double()[:, None, None] * (i[:, None] - j).abs()
                x.masked_fill_(~((j >= lo[:, None]) & (j < hi[:, None])), -math.inf)
                w = torch.softmax(x, -1).nan_to_num(0.0)               # rows that see nothing: zeros
                out[b, kv * rho:(kv + 1) * rho, t0:t1] = torch.einsum("htj,jd->htd", w, v[a:z])
    return out
