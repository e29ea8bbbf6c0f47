"""Paged attention at the edges of what it promises: tokens that see nothing beside numbers that are not finite."""
import math

import pytest
import torch

from test_paged_gpu import BF16, F32, Cache, draw, oracle, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def oal():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    oal.load_library()
    return oal


def put(c, j, value, b=0):
    """Key and value j of a sequence."""
    for pool in (c.Kp, c.Vp):
        pool[c.table[b, j // c.page].item(), :, j % c.page] = value


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,past", [(3, 30), (8, 40), (60, 30), (3, 2000), (8, 2000), (90, 2000), (300, 900)])
def test_tokens_that_see_nothing_beside_bad_numbers(oal, dtype, bad, T, past):
    """Of three tokens one sees nothing and gets zeros, one does not see the key that is bad, one does (and is not
    looked at); the keys in one piece and in several."""
    c = Cache(1, 2, [past], [T], 16, dtype, seed=101, fill=bad)
    Q = draw((1, 6, T, 64), dtype, 102, 1.5)
    first = torch.zeros(1, T, dtype=torch.int32)
    first[:, ::3], first[:, 1::3] = 1 << 28, past - 4
    put(c, past - 5, bad)
    Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, first=first.cuda())
    oal.oal_sync_status()
    assert (Y[:, :, ::3] == 0).all()
    put(c, past - 5, 0.0)
    want, size = oracle(c, Q, [T], first=first.cuda())
    off = (Y.double() - want).abs() - tolerance(dtype, want, size)
    assert (off[:, :, 1::3] <= 0).all()


def positive(n, Hkv, page, dtype, seed):
    """Pools whose values lie in 0.5 .. 1.5: a result is then as large as what its errors are counted in."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    K = torch.randn(n, Hkv, page, 64, device="cuda", generator=gen).to(dtype)
    return K, (0.5 + torch.rand(n, Hkv, page, 64, device="cuda", generator=gen)).to(dtype)


def same_within(dtype, a, b):
    """Two results of the same definition, each within its own tolerance."""
    b = b.double()
    return ((a.double() - b).abs() <= 2 * tolerance(dtype, b, b)).all()


def fastest(f):
    times = []
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("where", ["value", "both"])
@pytest.mark.parametrize("dtype,B,Hq,Hkv,T,past", [
    (BF16, 2, 16, 4, 8192, 0), (BF16, 2, 7, 1, 200, 60000), (BF16, 64, 32, 8, 4, 8000), (BF16, 2, 8, 2, 2, 131000),
    (F32, 2, 4, 2, 2500, 0), (F32, 32, 8, 2, 2, 6000)])
def test_one_bad_number_in_a_long_sequence(oal, dtype, B, Hq, Hkv, T, past, where):
    """A NaN in the first sequence, not seen by the tokens before it and by every third one behind it, whose documents
    start later: they and the other sequences do not change, and the call does not take many times as long."""
    page, most = 64, -(-(past + T) // 64)
    K, V = positive(B * most, Hkv, page, dtype, 131)
    Q = draw((B, Hq, T, 64), dtype, 132, 1.5)
    table = torch.arange(B * most, dtype=torch.int32, device="cuda").view(B, most)
    at, j = torch.full((B,), past, dtype=torch.int32, device="cuda"), past + T // 2
    first = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    first[0, T // 2 + 1::3] = j + 1
    sees_not = (torch.arange(T, device="cuda") < T // 2) | (first[0] > j)
    call = lambda: oal.oal_paged_attention(Q, K, V, table, at, first=first)
    want, clean = call(), fastest(call)
    V[j // page, :, j % page, 5] = math.nan
    if where == "both":
        K[j // page, :, j % page, 7] = math.nan
    got, bad = call(), fastest(call)
    oal.oal_sync_status()
    assert torch.equal(got[1:], want[1:])
    assert same_within(dtype, got[0][:, sees_not], want[0][:, sees_not])
    assert bad <= 12 * clean + 0.1, (bad, clean)


def test_rows_formed_again_outlast_no_wait(oal):
    """Rows of 2^18 keys in one piece that do not see a NaN which others of their tile see, under waits of half a
    millisecond: nothing waits for them, and the other sequences are as without it."""
    B, T, past, page = 8, 9984, 1 << 18, 128
    K, V = positive(9, 1, page, BF16, 141)
    Q = draw((B, 1, T, 64), BF16, 142, 1.5)
    table = 1 + torch.arange((past + T) // page, dtype=torch.int32, device="cuda") % 8
    table[0] = 0                                     # the first page is one of its own
    table = table.expand(B, -1).contiguous()
    first = torch.full((B, T), 8, dtype=torch.int32, device="cuda")
    first[0, 64:192:2] = 0
    at = torch.full((B,), past, dtype=torch.int32, device="cuda")
    call = lambda: oal.oal_paged_attention(Q, K, V, table, at, first=first)
    assert oal.oal_paged_attention_workspace_bytes(B, 1, 1, T, page, table.shape[1]) == 256
    want = call()
    V[0, :, 5] = math.nan
    oal.oal_debug_wait_test(1 << 20, 0)
    try:
        got = call()
        oal.oal_sync_status()
    finally:
        oal.oal_debug_wait_test(0, 0)
    assert torch.equal(got[1:], want[1:])
    rows = first[0] > 0
    assert same_within(BF16, got[0][:, rows], want[0][:, rows])


# ------------------------------------------------------------------ caps

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap", [100.0, 1e4, 1e6, 1e9])
@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_caps_far_above_the_scores(oal, dtype, cap, T):
    """Scores that a cap leaves nearly as they are.  (The tolerance knows no cap: such scores are as exact as without
    one: tanh(f) / f to 6e-8 and a few roundings, of scores up to 30 less than the 2e-5 of all scores.)"""
    c = Cache(2, 2, [300, 61], [T, T], 16, dtype, seed=111)
    Q = draw((2, 8, T, 64), dtype, 112, 1.5)
    Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, cap=cap)
    oal.oal_sync_status()
    want, size = oracle(c, Q, [T, T], cap=cap)
    assert ((Y.double() - want).abs() <= tolerance(dtype, want, size)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("T", [4, 40, 200])
def test_caps_near_some_scores_and_far_above_others(oal, dtype, slopes, T):
    """Every fifth token's scores reach the cap, its neighbours' do not."""
    c = Cache(1, 2, [333], [T], 16, dtype, seed=113)
    Q = draw((1, 8, T, 64), dtype, 114, 1.5)
    Q[:, :, ::5] *= 1e6
    kw = dict(cap=1e6, slopes=torch.linspace(0.0, 0.4, 8, device="cuda") if slopes else None)
    Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, **kw)
    oal.oal_sync_status()
    want, size = oracle(c, Q, [T], **kw)
    # (scores of up to 1e6 are off by 2^-24 of it and more: their tokens are not looked at)
    off = (Y.double() - want).abs() - tolerance(dtype, want, size)
    off[:, :, ::5] = 0
    assert (off <= 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap", [0.0, 30.0, 1e6])
@pytest.mark.parametrize("T", [5, 300])
def test_queries_behind_a_length_have_no_part(oal, dtype, cap, T):
    n = [T - T // 3, T // 2]
    c = Cache(2, 2, [200, 7], n, 16, dtype, seed=115, room=T // 16 + 1)
    Q = draw((2, 8, T, 64), dtype, 116, 1.5)
    got = []
    for rest in (0.0, 1e4, 1e30, math.nan, math.inf):
        for b in range(2):
            Q[b, :, n[b]:] = rest
        got.append(oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, cap=cap,
                                           lengths=torch.tensor(n, dtype=torch.int32, device="cuda")))
        oal.oal_sync_status()
    assert all(torch.equal(got[0], y) for y in got[1:])


# ------------------------------------------------------------------ nothing to see

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,T,past,page", [(2, 1, 0, 16), (8, 1, 100, 16), (8, 4, 100, 128), (16, 4, 250, 256),
                                                 (4, 40, 60, 128), (14, 300, 0, 16)])
def test_tiles_of_which_no_token_sees_anything(oal, dtype, Hq, T, past, page):
    """Keys in one piece where they are few: zeros, beside a sequence that is as it was."""
    c = Cache(2, 2, [past, past], [T, T], page, dtype, seed=151, fill=math.nan)
    Q = draw((2, Hq, T, 64), dtype, 152, 1.5)
    first = torch.zeros(2, T, dtype=torch.int32, device="cuda")
    want = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, first=first)
    for nothing in (1 << 28, 2 ** 31 - 1):
        first[0] = nothing
        Y = torch.full_like(Q, 7.0)
        oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, first=first, Y=Y)
        oal.oal_sync_status()
        assert (Y[0] == 0).all() and torch.equal(Y[1], want[1])


# ------------------------------------------------------------------ long sums

def repeated(oal, B, Hkv, rho, T, past, seed, page=128, distinct=8):
    """Mean relative error of attention over keys whose pages repeat (the definition then is a weighted softmax over
    one period), values of one sign."""
    per = page * distinct
    gen = torch.Generator(device="cuda").manual_seed(seed)
    K = torch.randn(distinct, Hkv, page, 64, device="cuda", generator=gen).to(BF16)
    V = (0.5 + torch.rand(distinct, Hkv, page, 64, device="cuda", generator=gen)).to(BF16)
    Q = (1.5 * torch.randn(B, Hkv * rho, T, 64, device="cuda", generator=gen)).to(BF16)
    n = -(-(past + T) // page)
    table = (torch.arange(n, device="cuda", dtype=torch.int32) % distinct).expand(B, n).contiguous()
    Y = oal.oal_paged_attention(Q, K, V, table, torch.full((B,), past, dtype=torch.int32, device="cuda"))
    oal.oal_sync_status()
    k, v = (x.transpose(0, 1).flatten(1, 2).double() for x in (K, V))
    off, j = [], torch.arange(per, device="cuda")
    for t in range(0, T, max(1, T // 64)):
        keys = past + t + 1
        q = Q[:, :, t].double().view(B, Hkv, rho, 64)
        s = 0.125 * torch.einsum("bhrd,hjd->bhrj", q, k)
        w = torch.exp(s - s.amax(-1, keepdim=True)) * (keys // per + (j < keys % per))
        y = torch.einsum("bhrj,hjd->bhrd", w, v) / w.sum(-1, keepdim=True)
        off.append(((Y[:, :, t].double().view(B, Hkv, rho, 64) - y) / y).flatten())
    return float(torch.cat(off).mean())


@pytest.mark.parametrize("B,Hkv,rho,T,past,most", [
    # The tensor cores cut what they add to an accumulator instead of rounding it: up to 2 2^-23 of it for every 16
    # keys (the accumulator's last bit and the products' lined up with it), which adds up over 16384 keys of a sum (a
    # chunk's) or 65536 (a token's) to 2.5e-4 and 9.8e-4.  The outputs' and weights' own roundings, independent in some
    # 32,768 of them, 2^-8 each: 6e-5 and less on the mean.
    (8, 1, 1, 9984, 1 << 20, 3.1e-4), (8, 1, 1, 9984, (1 << 18) + 77, 3.1e-4), (4, 2, 4, 4999, 1 << 19, 3.1e-4),
    (1217, 1, 4, 1, (1 << 20) - 1, 1.04e-3), (1217, 1, 4, 1, 1 << 18, 1.04e-3)])
def test_long_sums_of_one_sign(oal, B, Hkv, rho, T, past, most):
    assert abs(repeated(oal, B, Hkv, rho, T, past, 121)) <= most


# ------------------------------------------------------------------ layouts

@pytest.mark.parametrize("dtype,gap", [(F32, 4), (F32, 12), (BF16, 8)])
@pytest.mark.parametrize("T", [1, 100])
def test_pages_apart_by_any_multiple_of_16_bytes(oal, dtype, gap, T):
    c = Cache(1, 2, [70], [T], 16, dtype, seed=161)
    Q, K, V = (draw((1, h, T, 64), dtype, 162 + i, 1.5) for i, h in enumerate((4, 2, 2)))
    oal.oal_page_append(None, K, V, None, c.Kp, c.Vp, c.table, c.past)
    want = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past)
    shape, size = c.Kp.shape, c.Kp[0].numel()
    Kp, Vp = (torch.full((shape[0] * (size + gap),), math.nan, dtype=dtype, device="cuda")
              .as_strided(shape, (size + gap, *x.stride()[1:])) for x in (c.Kp, c.Vp))
    Kp.copy_(c.Kp), Vp.copy_(c.Vp)
    oal.oal_page_append(None, K, V, None, Kp, Vp, c.table, c.past)
    assert torch.equal(Kp, c.Kp) and torch.equal(Vp, c.Vp)
    assert torch.equal(oal.oal_paged_attention(Q, Kp, Vp, c.table, c.past), want)
    oal.oal_sync_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_tokens_of_one_place(oal, dtype):
    """Whatever is left there is of one or the other, and the rest of the cache as it was."""
    c = Cache(2, 2, [0, 0], [40, 40], 16, dtype, seed=171)
    c.table[1, 1] = c.table[0, 1]
    K = draw((2, 2, 40, 64), dtype, 172)
    before = c.Kp.clone()
    oal.oal_page_append(None, K, K, None, c.Kp, c.Vp, c.table, c.past)
    oal.oal_sync_status()
    at = c.table[0, 1].item()
    for pool in (c.Kp, c.Vp):
        assert ((pool[at] == K[0, :, 16:32]) | (pool[at] == K[1, :, 16:32])).all()
    for b in range(2):
        for i in (0, 2):
            rows = K[b, :, 16 * i:16 * i + 16]
            assert torch.equal(c.Kp[c.table[b, i].item(), :, :rows.shape[1]], rows)
    others = [i for i in range(c.n) if i not in c.table.flatten().tolist()]
    assert torch.equal(c.Kp[others], before[others])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,T,past,page,most", [
    (1, 14, 2, 1, 5000, 64, 128), (3, 8, 2, 4, 900, 16, 5000), (1, 4, 1, 300, 3000, 32, 2000), (2, 8, 8, 65, 100, 128, 40),
    (1, 2, 1, 1, 70000, 65536, 2), (1, 6, 2, 2000, 0, 64, 40), (9, 2, 2, 1, 250, 16, 17), (1300, 2, 1, 1, 50, 16, 20000)])
def test_workspace_is_not_overrun(oal, dtype, B, Hq, Hkv, T, past, page, most):
    """Exactly the size that is asked for, and numbers behind it that stay, whatever the masks."""
    c = Cache(B, Hkv, [past] * B, [T] * B, page, dtype, seed=181)
    c.table = torch.cat([c.table, torch.full((B, most - c.table.shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    Q = draw((B, Hq, T, 64), dtype, 182)
    need = oal.oal_paged_attention_workspace_bytes(B, Hq, Hkv, T, page, most, dtype=int(dtype is BF16))
    prefix = torch.full((B,), past + T, dtype=torch.int32, device="cuda")
    first = torch.full((B, T), past, dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(window=1), dict(window=100), dict(window=1000), dict(window=2 ** 31 - 1), dict(prefix=prefix),
               dict(prefix=prefix, window=300), dict(first=first), dict(first=first, window=300)):
        want = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, **kw)
        room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, workspace=room[:need], **kw)
        oal.oal_sync_status()
        assert torch.equal(Y, want) and (room[need:] == 0xA5).all()


@pytest.mark.parametrize("kind", ["none", "cap", "bias", "cap+bias", "window", "docs", "prefix", "all"])
def test_long_splits_as_short_ones(oal, kind):
    """6700 tokens on 36000 keys take splits of more than 16384 keys; 64 of them at a time, splits of fewer (compared
    with the definition above), to the tolerances of both.  Distances make the maximum grow all along the keys."""
    T, past, page = 6700, 36000, 64
    most = -(-(past + T) // page)
    K, V = positive(most, 2, page, BF16, 191)
    Q = draw((1, 8, T, 64), BF16, 192, 1.5)
    table = torch.randperm(most, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].cuda()
    kw, first = {}, None
    if "cap" in kind or kind == "all":
        kw["cap"] = 5.0
    if "bias" in kind or kind == "all":
        kw["slopes"] = torch.linspace(0.0, 2e-3, 8, device="cuda")
    if kind in ("window", "all"):
        kw["window"] = 30000
    if kind in ("prefix", "all"):
        kw["prefix"] = torch.tensor([past + T // 2], dtype=torch.int32, device="cuda")
    if kind in ("docs", "all"):
        t = torch.arange(T, dtype=torch.int32, device="cuda")[None]
        first = torch.where(t % 300 < 150, 7 * t, 11000)
    at = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    Y = oal.oal_paged_attention(Q, K, V, table, at(past), first=first, **kw)
    for t0 in (0, 1777, 3333, T - 64):
        part = slice(t0, t0 + 64)
        want = oal.oal_paged_attention(Q[:, :, part].contiguous(), K, V, table, at(past + t0), **kw,
                                       first=None if first is None else first[:, part].clone())
        oal.oal_sync_status()
        if "prefix" in kw and t0 + 64 < T // 2:      # (a prefix reaches as far as the sequence's keys)
            continue
        assert same_within(BF16, Y[:, :, part], want)
