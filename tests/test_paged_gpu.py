"""Rotary positions, the paged cache and its attention on the GPU, against the definitions in fp64."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}     # a rounding, relative
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def oal():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    oal.load_library()
    return oal


def draw(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=gen)).to(dtype).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotation

FREQ = [1e4 ** (-r / 32) for r in range(32)]


def turned(x, pos, freq, form, inverse=False):
    """x [B,H,T,64], pos [B,T,32]: fp64, and what its rounding errors are counted in: |x| + |y| of each pair."""
    a = pos.double() * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c, s = a.cos()[:, None], (-a if inverse else a).sin()[:, None]
    x = x.double()
    u, w = (x[..., :32], x[..., 32:]) if form == 0 else (x[..., 0::2], x[..., 1::2])
    out, size = (u * c - w * s, w * c + u * s), u.abs() + w.abs()
    if form == 0:
        return torch.cat(out, -1), torch.cat([size, size], -1)
    return torch.stack(out, -1).flatten(-2), torch.stack([size, size], -1).flatten(-2)


def check_turned(got, want, size):
    # cos and sin: one unit of sincospif (2^-24 of numbers up to 1) and the argument's rounding (an eighth of a turn,
    # pi / 4 2^-24); two products and a sum: 2 2^-24 of the pair; the reference's own angle: 2^-52 of up to 2^31 radians
    tol = size * (4 * 2.0 ** -24 + 2.0 ** -21 * (want.numel() == 0)) + want.abs() * HALF[got.dtype]
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("B,Hq,Hkv,T,lengths", [
    (1, 1, 1, 1, None), (1, 14, 2, 1, None), (3, 4, 4, 17, None), (64, 8, 2, 1, None), (2, 32, 8, 333, [333, 20]),
    (5, 3, 1, 15, [0, 1, 15, 14, 7]), (1, 4, 0, 100, None), (2, 7, 1, 16, None)])
def test_rope(oal, dtype, form, B, Hq, Hkv, T, lengths):
    Q = draw((B, Hq, T, 64), dtype, 1)
    K = draw((B, Hkv, T, 64), dtype, 2) if Hkv else None
    past = ints([(1000003 * b) % 4099 for b in range(B)])
    plan = oal.oal_rope_plan(FREQ)
    n = ints(lengths) if lengths else None
    Yq, Yk = torch.full_like(Q, 7.0), torch.full_like(K, 7.0) if Hkv else None
    oal.oal_rope(Q, K, plan, past=past, lengths=n, form=form, Yq=Yq, Yk=Yk)
    oal.oal_sync_status()
    pos = (past[:, None] + torch.arange(T, device="cuda"))[..., None].expand(B, T, 32)
    live = torch.arange(T, device="cuda") < (n[:, None] if lengths else T)
    live = live.expand(B, T)[:, None, :, None]
    for x, y in ((Q, Yq), (K, Yk)):
        if x is None:
            continue
        want, size = turned(x, pos, FREQ, form)
        check_turned(torch.where(live, y, 0), torch.where(live, want, 0), size)
        assert (torch.where(live, 7.0, y) == 7.0).all()
    # in place
    if lengths is None:
        q, k = Q.clone(), K.clone() if Hkv else None
        oal.oal_rope(q, k, plan, past=past, form=form, Yq=q, Yk=k)
        assert torch.equal(q, Yq) and (k is None or torch.equal(k, Yk))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rope_axes_far_positions_and_views(oal, dtype):
    B, Hq, Hkv, T = 2, 6, 2, 77
    qkv = draw((B, T, (Hq + 2 * Hkv) * 64 + 64), dtype, 3)[..., 64:].unflatten(-1, (-1, 64))
    Q, K = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    axes = [r % 3 for r in range(32)]
    gen = torch.Generator().manual_seed(4)
    positions = torch.randint(-2 ** 31, 2 ** 31, (3, B, T), generator=gen).to(torch.int32).cuda()
    positions[0, 0, 0], positions[1, 0, 0] = -2 ** 31, 2 ** 31 - 1
    plan = oal.oal_rope_plan(FREQ, axes)
    Yq, Yk = oal.oal_rope(Q, K, plan, positions=positions)
    oal.oal_sync_status()
    # angles of up to 2^31 radians in fp64 are off by 2^-22 at the most (their product's rounding): reduce exactly
    from fractions import Fraction
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    pos = positions[torch.tensor(axes)].permute(1, 2, 0).cpu()
    angle = torch.tensor([[[float((Decimal(int(p)) * Decimal(f)) % two_pi) for p, f in zip(row, FREQ)] for row in b]
                          for b in pos.tolist()], dtype=torch.float64, device="cuda")
    for x, y in ((Q, Yq), (K, Yk)):
        want, size = turned(x, angle, [1.0] * 32, 0)
        check_turned(y, want, size)
        assert y.is_contiguous()


@pytest.mark.parametrize("form", [0, 1])
def test_rope_gradient(oal, form):
    """The gradient of <dY, rope(Q)> is rope's inverse of dY: against the formula's and against differences."""
    Q, dY = draw((2, 3, 40, 64), F32, 5), draw((2, 3, 40, 64), F32, 6)
    plan, past = oal.oal_rope_plan(FREQ), ints([5, 900])
    dQ, _ = oal.oal_rope(dY, None, plan, past=past, form=form, inverse=True)
    pos = (past[:, None] + torch.arange(40, device="cuda"))[..., None].expand(2, 40, 32)
    q = Q.double().requires_grad_()
    turned(q, pos, FREQ, form)[0].backward(dY.double())
    check_turned(dQ, q.grad, turned(dY, pos, FREQ, form, True)[1])
    step = draw(Q.shape, F32, 7)
    f = lambda x: (turned(x, pos, FREQ, form)[0] * dY.double()).sum()
    slope = (f(Q.double() + 1e-3 * step.double()) - f(Q.double() - 1e-3 * step.double())) / 2e-3
    # linear in Q: the difference is exact but for fp64; dQ's errors are 4 2^-24 of each pair, summed with random signs at most
    assert abs(float(slope - (dQ.double() * step.double()).sum())) <= 5 * 2.0 ** -24 * float((step.abs() * dY.abs()).sum()) * 2


def test_rope_bad_axis_and_length_are_recorded(oal):
    Q, plan = draw((1, 2, 5, 64), F32, 8), oal.oal_rope_plan(FREQ, [3] * 32)
    positions = torch.zeros(2, 1, 5, dtype=torch.int32, device="cuda")
    Y, _ = oal.oal_rope(Q, None, plan, positions=positions)
    with pytest.raises(oal.OALError):
        oal.oal_sync_status()
    assert torch.equal(Y, Q)                       # counted as axis 0
    oal.oal_rope(Q, None, oal.oal_rope_plan(FREQ), lengths=ints([6]))
    with pytest.raises(oal.OALError):
        oal.oal_sync_status()
    oal.oal_sync_status()


# ------------------------------------------------------------------ cache

class Cache:
    """Pools, a table with the pages of each sequence in random order, lengths."""

    def __init__(self, B, Hkv, past, new, page, dtype, seed=0, room=0, joint=False, fill=None):
        most = max(-(-(a + b) // page) for a, b in zip(past, new)) + room
        n = B * most + 3
        gen = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(n, generator=gen)[:B * most].view(B, most).to(torch.int32).cuda()
        self.past, self.total, self.page, self.n = ints(past), [a + b for a, b in zip(past, new)], page, n
        if joint:
            pool = draw((n, 2, Hkv, page, 64), dtype, seed + 1)
            self.pool, self.Kp, self.Vp = pool, pool[:, 0], pool[:, 1]
        else:
            self.Kp, self.Vp = draw((n, Hkv, page, 64), dtype, seed + 1), draw((n, Hkv, page, 64), dtype, seed + 2)
        if fill is not None:                       # whatever lies behind a sequence's end
            for b in range(B):
                for j in range(self.total[b], most * page):
                    self.Kp[self.table[b, j // page].item(), :, j % page] = fill
                    self.Vp[self.table[b, j // page].item(), :, j % page] = fill

    def rows(self, pool, b, j0=0, j1=None):
        """Keys or values j0 .. j1 of a sequence, [Hkv, j, 64]."""
        j1 = self.total[b] if j1 is None else j1
        pages = self.table[b, j0 // self.page:-(-j1 // self.page)].long()
        x = pool[pages].transpose(0, 1).flatten(1, 2)
        return x[:, j0 % self.page:][:, :j1 - j0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,T,page,past,lengths,joint", [
    (1, 4, 2, 1, 16, [0], None, False), (1, 14, 2, 1, 64, [127], None, True), (3, 4, 4, 33, 16, [0, 15, 100], [33, 1, 0], False),
    (64, 8, 2, 1, 16, list(range(64)), None, False), (2, 6, 1, 300, 128, [5, 1000], [300, 299], True)])
def test_append(oal, dtype, B, Hq, Hkv, T, page, past, lengths, joint):
    new = lengths or [T] * B
    c = Cache(B, Hkv, past, [T] * B, page, dtype, seed=11, joint=joint)
    qkv = draw((B, T, Hq + 2 * Hkv, 64), dtype, 12)
    Q, K, V = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], 2))
    plan = oal.oal_rope_plan(FREQ)
    wantK, wantV = c.Kp.clone(), c.Vp.clone()
    Yq = oal.oal_page_append(Q, K, V, plan, c.Kp, c.Vp, c.table, c.past, lengths=ints(lengths) if lengths else None)
    oal.oal_sync_status()
    n = ints(lengths) if lengths else None
    q, k = oal.oal_rope(Q, K, plan, past=c.past, lengths=n)        # (tested above)
    assert torch.equal(Yq, q)
    for b in range(B):
        for t in range(new[b]):
            pg, row = c.table[b, (past[b] + t) // page].item(), (past[b] + t) % page
            wantK[pg, :, row], wantV[pg, :, row] = k[b, :, t], V[b, :, t]
    assert torch.equal(c.Kp, wantK) and torch.equal(c.Vp, wantV)
    # without a plan the rows go in as they are, and no queries
    oal.oal_page_append(None, K, V, None, c.Kp, c.Vp, c.table, c.past, lengths=n)
    for b in range(B):
        assert torch.equal(c.rows(c.Kp, b, past[b], past[b] + new[b]), K[b, :, :new[b]])
    # in 24-bit positions of its own
    positions = torch.randint(0, 1 << 24, (1, B, T), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    oal.oal_page_append(None, K, V, plan, c.Kp, c.Vp, c.table, c.past, positions=positions, lengths=n)
    k = oal.oal_rope(K, None, plan, positions=positions, lengths=n)[0]
    for b in range(B):
        assert torch.equal(c.rows(c.Kp, b, past[b], past[b] + new[b]), k[b, :, :new[b]])
    oal.oal_sync_status()


def test_append_without_a_place_is_recorded(oal):
    c = Cache(2, 2, [0, 0], [32, 32], 16, F32, seed=13)
    K = draw((2, 2, 32, 64), F32, 14)
    for past, table in (([0, 8], None), ([-1, 0], None), ([0, 0], -1), ([0, 0], c.n), ([0, 2 ** 31 - 1], None)):
        Kp, Vp, t = c.Kp.clone(), c.Vp.clone(), c.table.clone()
        if table is not None:
            t[1, 1] = table
        oal.oal_page_append(None, K, K, None, Kp, Vp, t, ints(past))
        with pytest.raises(oal.OALError):
            oal.oal_sync_status()
        want = c.Kp.clone()
        for b in range(2):
            for i in range(32):
                j = past[b] + i
                if 0 <= j < 32 and 0 <= t[b, j // 16] < c.n:
                    want[t[b, j // 16].item(), :, j % 16] = K[b, :, i]
        assert torch.equal(Kp, want)


# ------------------------------------------------------------------ attention

def oracle(c, Q, new, scale=0.125, cap=0.0, window=0, slopes=None, prefix=None, first=None):
    """fp64 [B,Hq,T,64], and sum_j softmax_j |v_j|, in which errors are counted."""
    B, Hq, T = Q.shape[:3]
    Hkv = c.Kp.shape[1]
    out = torch.zeros(2, B, Hq, T, 64, dtype=torch.float64, device="cuda")
    for b in range(B):
        past, n = c.past[b].item(), new[b]
        if n == 0:
            continue
        k, v = c.rows(c.Kp, b).double(), c.rows(c.Vp, b).double()
        i, j = torch.arange(past, past + n, device="cuda")[:, None], torch.arange(past + n, device="cuda")
        see = j <= i
        if prefix is not None:
            see = see | (j < prefix[b])
        if window:
            see = see & (j > i - window)
        if first is not None:
            see = see & (j >= first[b, :n, None])
        k, v = k.repeat_interleave(Hq // Hkv, 0), v.repeat_interleave(Hq // Hkv, 0)
        s = scale * Q[b, :, :n].double() @ k.transpose(1, 2)
        if cap:
            s = cap * torch.tanh(s / cap)
        if slopes is not None:
            s = s - slopes.double()[:, None, None] * (i - j).abs()
        s = torch.where(see, s, -math.inf)
        w = torch.where(see.any(-1, keepdim=True), torch.softmax(s, -1), 0.0)
        for x, y in zip(out, (v, v.abs())):
            # (a masked key's value has no part in the sum, whatever it is)
            finite = torch.isfinite(y)
            part = w @ torch.where(finite, y, 0.0)
            assert not (w.amax((0, 1))[~finite[0, :, 0]] > 0).any()
            x[b, :, :n] = part
    return out


def tolerance(dtype, want, size, cap=0.0):
    # bf16: the weights' rounding; the result's.  Scores: 64 fp32 products and sums (8 2^-24 of sizes up to 30, and a
    # cap's tanh, 4 2^-24 of it), exponentials 2^-22 of each weight, sums of weights
    d = 2e-5 + 4 * 2.0 ** -24 * cap + (HALF[dtype] if dtype is BF16 else 0.0)
    return size * d + want.abs() * HALF[dtype]


def check(oal, c, Q, new=None, **kw):
    T = Q.shape[2]
    Y = torch.full_like(Q, 7.0)
    n = ints(new) if new else None
    oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, lengths=n, Y=Y, **kw)
    oal.oal_sync_status()
    new = new or [T] * Q.shape[0]
    want, size = oracle(c, Q, new, **kw)
    live = (torch.arange(T, device="cuda") < ints(new)[:, None])[:, None, :, None]
    assert (torch.where(live, 7.0, Y) == 7.0).all()                       # rows behind a sequence stay
    got = torch.where(live, Y.double(), 0.0)
    off = (got - want).abs() - tolerance(Q.dtype, want, size, kw.get("cap", 0.0))
    assert (off <= 0).all(), (float(off.max()), [int(x) for x in (off == off.max()).nonzero()[0]])
    return Y


SHAPES = [  # B, Hq, Hkv, T, past, page, lengths
    (1, 1, 1, 1, [0], 16, None), (1, 2, 1, 1, [1], 16, None), (2, 14, 2, 1, [127, 128], 64, None),
    (1, 16, 1, 1, [4095], 16, None), (3, 20, 1, 1, [31, 32, 500], 32, None), (1, 128, 1, 1, [77], 16, None),
    (2, 14, 2, 1, [3000, 20000], 128, None), (5, 8, 8, 1, [0, 1, 2, 3, 4], 16, [1, 0, 1, 1, 0]),
    (2, 8, 2, 5, [1000, 17], 16, [5, 2]), (2, 7, 1, 3, [64, 255], 64, None), (1, 4, 4, 2, [2000], 256, None),
    (1, 4, 1, 33, [0], 16, None), (2, 4, 2, 64, [64, 0], 64, None), (1, 5, 1, 65, [63], 32, None),
    (2, 14, 2, 129, [0, 333], 16, [129, 7]), (1, 3, 3, 257, [0], 128, None), (3, 4, 2, 300, [0, 1, 700], 32, [300, 0, 255]),
    (1, 2, 1, 1000, [24], 64, None), (1, 28, 4, 200, [5000], 128, None), (1, 128, 1, 5, [300], 16, None),
    (1, 100, 2, 9, [129], 16, None), (1, 1, 1, 515, [0], 65536, None)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,T,past,page,lengths", SHAPES)
def test_attention(oal, dtype, B, Hq, Hkv, T, past, page, lengths):
    c = Cache(B, Hkv, past, lengths or [T] * B, page, dtype, seed=21, fill=math.nan if page < 1000 else None)
    check(oal, c, draw((B, Hq, T, 64), dtype, 22, 1.5), lengths)


MASKS = ["cap", "small cap", "window", "bias", "docs", "prefix", "window+prefix", "cap+bias", "all", "nothing"]


def masks(kind, B, Hq, T, past, lengths):
    new = lengths or [T] * B
    kw = {}
    if "cap" in kind or kind == "all":
        kw["cap"] = 30.0 if "small" in kind else 3.0      # (of small scores: their share of the cap is)
    if "window" in kind or kind == "all":
        kw["window"] = 50
    if "bias" in kind or kind == "all":
        kw["slopes"] = torch.linspace(0.0, 0.4, Hq, device="cuda")
    if kind in ("docs", "all"):
        t = torch.arange(T)[None] + torch.tensor(past)[:, None]
        start = torch.rand(B, T, generator=torch.Generator().manual_seed(5)) < 0.05
        kw["first"] = torch.where(start, t, 0).cummax(1).values.to(torch.int32).cuda()
    if "prefix" in kind or kind == "all":
        kw["prefix"] = ints([a + n // 2 + 3 for a, n in zip(past, new)])
    if kind == "nothing":                           # every third token sees nothing
        first = torch.zeros(B, T, dtype=torch.int32)
        first[:, ::3] = 1 << 29
        kw["first"] = first.cuda()
    return kw


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("B,Hq,Hkv,T,past,page,lengths", [
    (2, 14, 2, 1, [300, 40], 16, None), (3, 8, 2, 4, [100, 0, 777], 32, [4, 3, 1]), (2, 4, 2, 70, [0, 190], 16, [70, 33]),
    (1, 6, 2, 400, [250], 64, None), (2, 3, 1, 260, [0, 3000], 128, None)])
def test_masks(oal, dtype, kind, B, Hq, Hkv, T, past, page, lengths):
    c = Cache(B, Hkv, past, lengths or [T] * B, page, dtype, seed=23, fill=math.nan)
    check(oal, c, draw((B, Hq, T, 64), dtype, 24, 1.5), lengths, **masks(kind, B, Hq, T, past, lengths))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,T", [(8, 1500), (2, 1100), (14, 700)])
@pytest.mark.parametrize("turn", [0, 1])
def test_documents_of_unequal_lengths(oal, dtype, Hq, T, turn):
    """Neighbouring tiles of rows whose keys begin far apart, the first or the second one's earlier; tiles that see
    nothing between others."""
    c = Cache(1, 2, [40], [T], 32, dtype, seed=61, fill=math.nan)
    Q = draw((1, Hq, T, 64), dtype, 62, 1.5)
    for width in (32, 96, 128, 18):
        t = torch.arange(T)
        odd = t // width % 2 == turn
        check(oal, c, Q, first=torch.where(odd, 0, (t + 40 - t % width).clamp(min=0)).to(torch.int32)[None].cuda())
        check(oal, c, Q, first=torch.where(odd, 0, 1 << 28).to(torch.int32)[None].cuda())
        check(oal, c, Q, first=torch.where(t % (2 * width) == (2 * width - 1 if turn else 0), t + 40, 1 << 28).to(torch.int32)[None].cuda())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("T,past", [(1, 5000), (6, 900), (90, 4000), (300, 200)])
def test_masked_keys_have_no_part(oal, dtype, bad, T, past):
    """Infinities and NaN in keys and values that a row's window or document leaves out, though others of its tile
    or page see them: those that see them are not looked at, the others are as if they were not there."""
    B, Hq, Hkv, page = 1, 4, 2, 32
    c = Cache(B, Hkv, [past], [T], page, dtype, seed=25, fill=bad)
    Q = draw((B, Hq, T, 64), dtype, 26, 1.5)
    first = torch.full((B, T), past - 40, dtype=torch.int32)
    first[:, T // 2:] = past - 8
    for j in (past - 41, past - 9, past - 100, 3):
        pg = c.table[0, j // page].item()
        c.Kp[pg, :, j % page] = bad
        c.Vp[pg, :, j % page] = bad
    seen = torch.zeros(T, dtype=torch.bool)
    seen[:T // 2] = True                             # key past - 9
    first = first.cuda()
    Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, first=first)
    oal.oal_sync_status()
    clean = Cache(B, Hkv, [past], [T], page, dtype, seed=25, fill=0.0)
    for j in (past - 9,):                            # of the rows that do not see it
        pg = clean.table[0, j // page].item()
        clean.Kp[pg, :, j % page] = 0
        clean.Vp[pg, :, j % page] = 0
    want, size = oracle(clean, Q, [T], first=first)
    rows = (~seen).nonzero().flatten().cuda()
    off = (Y.double() - want).abs() - tolerance(dtype, want, size)
    assert (off[:, :, rows] <= 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 7, 140])
def test_pages(oal, dtype, T):
    """Pages before the window need not exist; a bad page among the visible ones is recorded, and nothing else breaks."""
    past = 700
    c = Cache(2, 2, [past, 90], [T, T], 16, dtype, seed=27, fill=math.nan)
    Q = draw((2, 4, T, 64), dtype, 28)
    want = check(oal, c, Q, window=100)
    c.table[0, :(past - 99) // 16] = -1
    Y = torch.full_like(Q, 7.0)
    oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, window=100, Y=Y)
    oal.oal_sync_status()
    assert torch.equal(Y, want)
    for bad in (-1, c.n, 2 ** 31 - 1, -2 ** 31):
        c.table[0, past // 16 - 1] = bad
        Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, window=100)
        with pytest.raises(oal.OALError):
            oal.oal_sync_status()
        assert torch.equal(Y[1], want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 40])
def test_bad_past_and_lengths_are_recorded(oal, dtype, T):
    c = Cache(2, 2, [60, 60], [T, T], 16, dtype, seed=29)
    Q = draw((2, 4, T, 64), dtype, 30)
    want = check(oal, c, Q)
    for past, lengths in (([60, -1], None), ([60, 1 << 20], None), ([60, 2 ** 31 - 1], None), ([60, 60], [T, -1]), ([60, 60], [T, T + 1])):
        Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, ints(past), lengths=ints(lengths) if lengths else None)
        with pytest.raises(oal.OALError):
            oal.oal_sync_status()
        assert torch.equal(Y[0], want[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(oal, dtype):
    """Scores of thousands, rising and falling along the keys, of one sign: the running maximum."""
    for T, past in ((1, 900), (150, 333)):
        c = Cache(1, 1, [past], [T], 16, dtype, seed=31)
        ramp = torch.linspace(-40.0, 40.0, past + T, device="cuda").to(dtype)
        for up in (1.0, -1.0):
            for j in range(past + T):
                c.Kp[c.table[0, j // 16].item(), :, j % 16] = up * ramp[j]
            Q = torch.full((1, 2, T, 64), 1.0, dtype=dtype, device="cuda")
            Q[:, 1] = -1.0
            Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past)
            want, size = oracle(c, Q, [T])
            # scores of up to 320.  bf16: the sums of 64 equal products are exact (14 bits), the scale, the product by
            # it and the difference to the maximum round by 2^-24 each, of up to 460 in units of the base 2: 9e-5.
            # fp32: a sum of i products x of 24 bits rounds by 2^-24 i x, all 64 by 2080 2^-24 x at most, which is
            # 6.2e-4 of a score for x = 40 and the scale 1 / 8; a weight is off by that of two scores.
            d = 1.3e-3 if dtype is F32 else 2e-4 + HALF[dtype]
            assert ((Y.double() - want).abs() <= size * d + want.abs() * HALF[dtype]).all()


def test_offsets_behind_two_to_the_31(oal):
    """A pool of more than 2^31 elements, whose last pages are in use."""
    n, page = 18000, 1024
    pool = torch.empty(n, 2, 1, page, 64, dtype=BF16, device="cuda")     # 4.7 GB
    c = Cache(1, 1, [1500], [600], page, BF16, seed=33)
    c.table = ints([[n - 1, 5, n - 2]])
    small = draw((3, 2, 1, page, 64), BF16, 34)
    for i, at in enumerate(c.table[0].tolist()):
        pool[at] = small[i]
    c.Kp, c.Vp = pool[:, 0], pool[:, 1]
    check(oal, c, draw((1, 2, 600, 64), BF16, 35))
    K = draw((1, 1, 600, 64), BF16, 37)
    oal.oal_page_append(None, K, K, None, c.Kp, c.Vp, c.table, c.past)
    assert torch.equal(c.rows(c.Vp, 0, 1500, 2100), K[0])
    c.past, c.total = ints([2099]), [2100]
    check(oal, c, draw((1, 2, 1, 64), BF16, 36))


@pytest.mark.parametrize("Hq", [1, 2])
def test_sixteen_million_tokens(oal, Hq):
    """More tiles than a grid's second and third dimension hold; everyone sees itself, the last ones one key more."""
    T, page = (1 << 24) + 300, 65536
    n = -(-T // page)
    gen = torch.Generator(device="cuda").manual_seed(63)
    V = torch.randn(n, 1, page, 64, device="cuda", dtype=BF16, generator=gen)
    K = torch.randn(n, 1, page, 64, device="cuda", dtype=BF16, generator=gen)
    Q = torch.randn(1, Hq, T, 64, device="cuda", dtype=BF16, generator=gen)
    table = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    Y = oal.oal_paged_attention(Q, K, V, table, ints([0]), window=1)
    oal.oal_sync_status()
    for h in range(Hq):                            # a weight of 1: the values themselves
        assert torch.equal(Y[0, h], V.view(-1, 64)[:T])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,past", [(1, 9000), (20, 300), (300, 1000)])
def test_same_bits_twice_and_more_room(oal, dtype, T, past):
    """The same call gives the same bits; a table with room for more may split the keys otherwise."""
    c = Cache(1, 2, [past], [T], 16, dtype, seed=38)
    Q = draw((1, 8, T, 64), dtype, 39)
    a = check(oal, c, Q)
    b = check(oal, c, Q)
    assert torch.equal(a, b)
    c.table = torch.cat([c.table, torch.full((1, 3000), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    check(oal, c, Q)


def test_streams_graphs_and_two_calls_at_once(oal):
    dtype = BF16
    cs = [Cache(2, 2, [700, 64], [T, T], 16, dtype, seed=40 + T) for T in (1, 5, 200)]
    qs = [draw((2, 8, T, 64), dtype, 50 + T) for T in (1, 5, 200)]
    want = [check(oal, c, q) for c, q in zip(cs, qs)]
    call = lambda c, q, **kw: oal.oal_paged_attention(q, c.Kp, c.Vp, c.table, c.past, **kw)
    # another stream, the current one busy
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        a = a @ a * 1e-2
    got = [call(c, q, stream=side) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[call(c, q, stream=s) for c, q in zip(cs, qs)] for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for row in got for x, y in zip(row, want))
    # captured, replayed on other inputs: the length grows by a token
    c, q = cs[0], qs[0].clone()
    K = draw((2, 2, 1, 64), dtype, 60)
    plan = oal.oal_rope_plan(FREQ)
    Y, Yq = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.empty(oal.oal_paged_attention_workspace_bytes(2, 8, 2, 1, 16, c.table.shape[1]), dtype=torch.uint8, device="cuda")
    def step():
        oal.oal_page_append(q, K, K, plan, c.Kp, c.Vp, c.table, c.past, Yq=Yq)
        call(c, Yq, Y=Y, workspace=ws)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(3):
        q.copy_(draw(q.shape, dtype, 70 + t))
        K.copy_(draw(K.shape, dtype, 80 + t))
        c.past.copy_(ints([701 + t, 65 + t]))
        graph.replay()
        torch.cuda.synchronize()
        c.total = [702 + t, 66 + t]
        w, size = oracle(c, Yq, [1, 1])
        assert ((Y.double() - w).abs() <= tolerance(dtype, w, size)).all()
    oal.oal_sync_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_serving_run(oal, dtype):
    """Two prompts in chunks of unequal lengths, a fork of their pages, tokens one by one and drafted ones."""
    B, Hq, Hkv, page, most = 2, 6, 2, 16, 24
    n = B * most
    pool = torch.full((n, 2, Hkv, page, 64), math.nan, dtype=dtype, device="cuda")
    table = torch.randperm(n, generator=torch.Generator().manual_seed(1)).view(B, most).to(torch.int32).cuda()
    plan = oal.oal_rope_plan(FREQ)
    seen = [[torch.zeros(Hkv, 0, 64, dtype=dtype, device="cuda") for _ in range(2)] for _ in range(B)]
    past = [0, 0]
    for step, new in enumerate([[100, 37], [1, 1], [5, 5], [1, 0], [130, 64], [1, 1]]):
        T = max(new)
        Q, K, V = (draw((B, h, T, 64), dtype, 100 * step + h + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        at, lengths = ints(past), ints(new)
        q = oal.oal_page_append(Q, K, V, plan, pool[:, 0], pool[:, 1], table, at, lengths=lengths)
        if step == 2:                                 # the second sequence goes on in copies of its pages
            old = table[1].tolist()
            fresh = [x for x in range(n) if x not in table[0].tolist()][::-1]
            table[1] = ints(fresh)
            table_map = torch.arange(n, dtype=torch.int32)
            for a, z in zip(fresh, old):
                table_map[a] = z
            oal.oal_state_remap(pool, table_map.cuda())
        Y = oal.oal_paged_attention(q, pool[:, 0], pool[:, 1], table, at, lengths=lengths, scale=0.2)
        oal.oal_sync_status()
        pos = (at[:, None] + torch.arange(T, device="cuda"))[..., None].expand(B, T, 32)
        k = turned(K, pos, FREQ, 0)[0].to(dtype)
        for b in range(B):
            if new[b] == 0:
                continue
            seen[b] = [torch.cat([x, y[b, :, :new[b]]], 1) for x, y in zip(seen[b], (k, V))]
            kk, vv = (x.double().repeat_interleave(Hq // Hkv, 0) for x in seen[b])
            s = 0.2 * turned(Q, pos, FREQ, 0)[0][b, :, :new[b]].to(dtype).double() @ kk.transpose(1, 2)
            j = torch.arange(past[b] + new[b], device="cuda")
            w = torch.softmax(torch.where(j <= j[past[b]:, None], s, -math.inf), -1)
            want, size = w @ vv, w @ vv.abs()
            # a rotated row may be rounded to the other neighbour than the reference's: fp32 1e-6, bf16 a step now and
            # then, which moves a score by 2^-8 |q k| scale at most (2^-8 0.2 4 4 of a few elements)
            d = 4e-5 if dtype is F32 else 2.0 ** -8 + 2.0 ** -8 * 3.2
            assert ((Y[b, :, :new[b]].double() - want).abs() <= size * d + want.abs() * HALF[dtype]).all()
            past[b] += new[b]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotations_feed_the_other_layers(oal, dtype):
    """The quadratic and the gated layer on what a rotation has just written, and paged attention on what an append
    has: the same bits as with a pause between the calls."""
    B, Hq, Hkv, T = 2, 4, 2, 300
    L = torch.tril(0.2 * torch.randn(Hq, 3, 3, generator=torch.Generator().manual_seed(1))).cuda() + 0.6 * torch.eye(3, device="cuda")
    group = torch.ones(Hq, 64, dtype=torch.int32, device="cuda")
    group[:, :5] = 2
    tables = oal.oal_expand_coeffs(L, group, 1e-6, oal.OAL_STATE_PACKED)
    plan, gate = oal.oal_rope_plan(FREQ), torch.full((B, Hkv, T), -0.05, device="cuda")
    c = Cache(B, Hkv, [10, 70], [T, T], 16, dtype, seed=90)
    Yq, Yk = torch.empty(B, Hq, T, 64, dtype=dtype, device="cuda"), torch.empty(B, Hkv, T, 64, dtype=dtype, device="cuda")
    layers = [lambda V: oal.oal_prefill(Yq, Yk, V, L, group, 1e-6, *tables, oal.OAL_STATE_PACKED),
              lambda V: oal.oal_gated_prefill(Yq, Yk, V, gate),
              lambda V: [oal.oal_paged_attention(Yq, c.Kp, c.Vp, c.table, c.past)]]
    for step in range(4):
        Q, K, V = (draw((B, h, T, 64), dtype, 7 * step + i, 0.7) for i, h in enumerate((Hq, Hkv, Hkv)))
        for i, layer in enumerate(layers):
            got = []
            for pause in (False, True):
                Yq.fill_(9.0), Yk.fill_(9.0)
                torch.cuda.synchronize()
                if i < 2:
                    oal.oal_rope(Q, K, plan, past=c.past, Yq=Yq, Yk=Yk)
                else:
                    c.Kp.fill_(9.0), c.Vp.fill_(9.0)
                    oal.oal_page_append(Q, K, V, plan, c.Kp, c.Vp, c.table, c.past, Yq=Yq)
                if pause:
                    torch.cuda.synchronize()
                got.append(layer(V))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(*got))
    oal.oal_sync_status()


@pytest.mark.parametrize("T", [1, 12, 300])
def test_graphs_with_workspaces_of_their_own(oal, T):
    """Two captured calls that split their keys and were given no workspace, replayed at once on two streams, eager
    calls in between."""
    cs = [Cache(1, 2, [past], [T], 32, BF16, seed=91 + past) for past in (9000, 7001)]
    qs = [draw((1, 8, T, 64), BF16, 95 + i) for i in range(2)]
    want = [check(oal, c, q) for c, q in zip(cs, qs)]
    ys, graphs = [torch.zeros_like(q) for q in qs], []
    side = torch.cuda.Stream()
    for c, q, y in zip(cs, qs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                oal.oal_paged_attention(q, c.Kp, c.Vp, c.table, c.past, Y=y)
        graphs.append(graph)
    assert oal.oal_paged_attention_workspace_bytes(1, 8, 2, T, 32, cs[0].table.shape[1]) > 256
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = oal.oal_paged_attention(qs[0], cs[0].Kp, cs[0].Vp, cs[0].table, cs[0].past)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
    oal.oal_sync_status()


def test_append_in_place(oal):
    """The turned queries may take the place of the queries."""
    c = Cache(2, 2, [3, 40], [50, 50], 16, BF16, seed=99)
    Q, K, V = (draw((2, h, 50, 64), BF16, 99 + i) for i, h in enumerate((6, 2, 2)))
    plan = oal.oal_rope_plan(FREQ)
    want = oal.oal_page_append(Q, K, V, plan, c.Kp, c.Vp, c.table, c.past)
    pools = c.Kp.clone(), c.Vp.clone()
    oal.oal_page_append(Q, K, V, plan, c.Kp, c.Vp, c.table, c.past, Yq=Q)
    assert torch.equal(Q, want) and torch.equal(c.Kp, pools[0]) and torch.equal(c.Vp, pools[1])
    oal.oal_sync_status()
