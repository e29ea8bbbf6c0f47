"""Gated recurrence (prefill, decode step, backward) and state remap on a GPU,
against the definitions in 64 bits, one token after another.

Tolerances, rel-L2 over a tensor:
  * fp32 inputs: every output is a sum of at most a few thousand products in
    fp32; independent roundings grow like sqrt(n) 2^-24, 4e-6 at n = 4096;
    1e-5 leaves room for the few sums in a row that an output passes.
  * bf16 inputs, bf16 outputs: three roundings to bf16 (a score, a state, the
    result), each off by at most 2^-8 of its value: 3 * 2^-8 = 1.2e-2.
  * bf16 inputs, fp32 outputs: the states and their gradients are sums of fp32
    products like those of fp32 inputs, 1e-5; 2e-5 allows a factor held as two
    bf16 terms (2^-16).  dg is a sum of four parts, in which states count as
    two such terms: 2 * 2^-16 < 3.1e-5, 4e-5 with the sums.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 0.125
OUT = {torch.float32: 1e-5, torch.bfloat16: 3 * 2.0 ** -8}
STATE = {torch.float32: 1e-5, torch.bfloat16: 2e-5}
DG = {torch.float32: 1e-5, torch.bfloat16: 4e-5}
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def oal():
    from grouped_quadratic_gb300 import build, oal as binding
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.load_library()
    return binding


class Case:
    def __init__(self, dtype, B, Hq, Hkv, T, seed=0, cut=0.0, span=30.0, lengths=None):
        gen = torch.Generator().manual_seed(1000 + seed)
        n = lambda *s: torch.randn(*s, generator=gen)
        self.dtype, self.B, self.Hq, self.Hkv, self.T = dtype, B, Hq, Hkv, T
        self.Q, self.dY = (n(B, Hq, T, 64).to(dtype).cuda() for _ in range(2))
        self.K, self.V = (n(B, Hkv, T, 64).to(dtype).cuda() for _ in range(2))
        self.g = torch.nn.functional.logsigmoid(n(B, Hkv, T) + math.log(span))
        if cut:
            self.g[torch.rand(B, Hkv, T, generator=gen) < cut] = -math.inf
        self.g = self.g.cuda()
        self.state0, self.dstate = (n(B, Hkv, 64, 64).cuda() for _ in range(2))
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()

    def rows(self, like):
        """Which rows of a [B, H, T, ...] tensor are inside their sequence."""
        n = self.lengths.tolist() if self.lengths is not None else [self.T] * self.B
        m = torch.tensor([[t < x for t in range(self.T)] for x in n], dtype=torch.bool).cuda()
        return m.view(self.B, 1, self.T, *[1] * (like.dim() - 3)).expand_as(like)


def oracle(c, state0=None, dstate=None, backward=False, scale=SCALE):
    """fp64: Y and the last state, or dQ, dK, dV, dg, dstate0."""
    B, Hkv, T, rho = c.B, c.Hkv, c.T, c.Hq // c.Hkv
    n = c.lengths.cpu() if c.lengths is not None else torch.full((B,), T)
    Q, K, V, g, dY = (x.double().cpu() for x in (c.Q, c.K, c.V, c.g, c.dY))
    Q, dY = Q.view(B, Hkv, rho, T, 64), dY.view(B, Hkv, rho, T, 64)
    S = torch.zeros(B, Hkv, 64, 64, dtype=torch.float64) if state0 is None else state0.double().cpu()
    R = torch.zeros_like(S) if dstate is None else dstate.double().cpu()
    Y, dQ = torch.zeros_like(Q), torch.zeros_like(Q)
    dK, dV, dg = torch.zeros_like(K), torch.zeros_like(V), torch.zeros_like(g)
    path = [S]
    for t in range(T):
        on = t < n                                         # the sequences that have this token
        new = g[:, :, t].exp()[..., None, None] * S + K[:, :, t, :, None] * V[:, :, t, None, :]
        S = torch.where(on.view(B, 1, 1, 1), new, S)
        path.append(S if backward else None)
        Y[on, :, :, t] = scale * (Q[on, :, :, t] @ S[on])
        dQ[on, :, :, t] = scale * (dY[on, :, :, t] @ S[on].transpose(-1, -2))
    if not backward:
        return Y.view(B, c.Hq, T, 64), S
    for t in reversed(range(T)):
        on = t < n
        new = R + scale * Q[:, :, :, t].transpose(-1, -2) @ dY[:, :, :, t]
        dK[on, :, t] = (new @ V[:, :, t, :, None])[on, ..., 0]
        dV[on, :, t] = (new.transpose(-1, -2) @ K[:, :, t, :, None])[on, ..., 0]
        new = g[:, :, t].exp()[..., None, None] * new
        dg[on, :, t] = (new * path[t]).sum((-1, -2))[on]
        R = torch.where(on.view(B, 1, 1, 1), new, R)
    return dQ.view(B, c.Hq, T, 64), dK, dV, dg, R


def rel(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(got).all()
    return float((got - want).norm() / max(float(want.norm()), 1e-30))


def run_forward(oal, c, cont=False, **kw):
    state = c.state0.clone() if cont else torch.full_like(c.state0, math.nan)
    Y = torch.full_like(c.Q, 7.0)
    oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, SCALE, lengths=c.lengths, state=state,
                          continue_from_state=cont, Y=Y, **kw)
    oal.oal_sync_status()
    return Y, state


def check_forward(oal, c, cont):
    Y, state = run_forward(oal, c, cont)
    want, S = oracle(c, c.state0 if cont else None)
    inside = c.rows(Y)
    assert (Y[~inside] == 7.0).all()                       # rows behind a sequence stay
    assert rel(torch.where(inside, Y, 0), want) <= OUT[c.dtype]
    assert rel(state, S) <= STATE[c.dtype]


def check_backward(oal, c, cont):
    out = [torch.full_like(x, 7.0) for x in (c.Q, c.K, c.V, c.g)]
    got = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=c.lengths,
                                 state0=c.state0 if cont else None, dstate=c.dstate if cont else None,
                                 dQ=out[0], dK=out[1], dV=out[2], dg=out[3])
    oal.oal_sync_status()
    want = oracle(c, c.state0 if cont else None, c.dstate if cont else None, backward=True)
    tol = [OUT[c.dtype]] * 3 + [DG[c.dtype], STATE[c.dtype]]
    for name, a, w, t in zip(("dQ", "dK", "dV", "dg", "dstate0"), got, want, tol):
        if name != "dstate0":
            assert (a[~c.rows(a)] == 7.0).all(), name
            a = torch.where(c.rows(a), a, 0)
        if w.norm() == 0:                                  # one token from no state
            assert (a == 0).all(), name
        else:
            assert rel(a, w) <= t, (name, rel(a, w))


SHAPES = [  # B, Hq, Hkv, T, cut, lengths, cont
    (1, 1, 1, 1, 0.0, None, False), (1, 1, 1, 1, 0.0, None, True), (2, 3, 3, 2, 0.3, None, True),
    (1, 2, 1, 63, 0.0, None, False), (1, 2, 2, 64, 0.0, None, True), (2, 2, 1, 65, 0.05, None, True),
    (1, 7, 1, 128, 0.0, None, False), (1, 14, 2, 129, 0.02, None, True), (2, 10, 2, 191, 0.0, [191, 17], False),
    (4, 4, 2, 333, 0.01, [0, 1, 333, 64], True), (1, 4, 4, 640, 0.0, None, False),
    (3, 9, 1, 257, 1.0, [257, 256, 3], True), (1, 8, 1, 2050, 0.001, None, True),
    # segments of several chunks: one segment a sequence, and two
    (160, 3, 3, 170, 0.003, [170, 169, 128, 129, 5, 0, 64, 65] * 20, True), (60, 10, 2, 400, 0.003, None, False)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,T,cut,lengths,cont", SHAPES)
def test_prefill(oal, dtype, B, Hq, Hkv, T, cut, lengths, cont):
    check_forward(oal, Case(dtype, B, Hq, Hkv, T, seed=T + B, cut=cut, lengths=lengths), cont)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,T,cut,lengths,cont", SHAPES)
def test_backward(oal, dtype, B, Hq, Hkv, T, cut, lengths, cont):
    check_backward(oal, Case(dtype, B, Hq, Hkv, T, seed=T + B + 1, cut=cut, lengths=lengths), cont)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [0.0, -1e-4, -3.0, -60.0, -103.0, -104.0, -2e38, -math.inf])
def test_one_gate_everywhere(oal, dtype, gate):
    c = Case(dtype, 1, 4, 2, 200, seed=3)
    c.g = torch.full_like(c.g, gate)
    check_forward(oal, c, True)
    check_backward(oal, c, True)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_gates_of_very_different_size(oal, dtype):
    """A large drop must not cost the digits of the small ones behind it."""
    c = Case(dtype, 1, 4, 2, 300, seed=4, span=500.0)
    c.g[:, :, 5::23] = -90.0
    c.g[:, :, 11::31] = -40.0
    check_forward(oal, c, True)
    check_backward(oal, c, True)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_growing_gates(oal, dtype):
    c = Case(dtype, 1, 4, 2, 150, seed=5)
    c.g = c.g.abs() * 0.2
    check_forward(oal, c, True)
    check_backward(oal, c, True)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_many_segments(oal, dtype):
    c = Case(dtype, 1, 2, 1, 6000, seed=6, span=2000.0)
    check_forward(oal, c, True)
    check_backward(oal, c, True)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_padding_is_not_read(oal, dtype):
    lengths = [70, 0, 200]
    c = Case(dtype, 3, 4, 2, 200, seed=7, lengths=lengths)
    Y0, S0 = run_forward(oal, c, True)
    G0 = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=c.lengths, state0=c.state0)
    for b, n in enumerate(lengths):
        for x in (c.Q, c.K, c.V, c.g, c.dY):
            x[b, :, n:] = math.nan
    Y1, S1 = run_forward(oal, c, True)
    G1 = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=c.lengths, state0=c.state0)
    oal.oal_sync_status()
    assert torch.equal(Y0, Y1) and torch.equal(S0, S1)
    assert all(torch.equal(a, b) for a, b in zip(G0, G1))


def test_made_here_rows_are_zero(oal):
    c = Case(torch.bfloat16, 2, 2, 1, 100, seed=8, lengths=[40, 100])
    Y, _ = oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, lengths=c.lengths)
    G = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, lengths=c.lengths)
    oal.oal_sync_status()
    for x in (Y,) + G[:4]:
        assert (x[0, :, 40:] == 0).all()


@pytest.mark.parametrize("bad", [-1, 51])
def test_length_out_of_range_is_recorded(oal, bad):
    c = Case(torch.float32, 2, 2, 1, 50, seed=9)
    lengths = torch.tensor([50, bad], dtype=torch.int32).cuda()
    Y, S = oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, SCALE, lengths=lengths)
    with pytest.raises(oal.OALError) as e:
        oal.oal_sync_status()
    assert e.value.status == oal.OAL_ERR_INVALID_ARG
    oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=lengths)
    with pytest.raises(oal.OALError):
        oal.oal_sync_status()
    oal.oal_sync_status()
    c.lengths = torch.tensor([50, max(0, min(50, bad))], dtype=torch.int32).cuda()   # clamped
    want, S64 = oracle(c)
    assert rel(Y, want) <= OUT[c.dtype] and rel(S, S64) <= STATE[c.dtype]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_empty_sequences(oal, dtype):
    c = Case(dtype, 2, 2, 1, 0, seed=10)
    _, S = run_forward(oal, c, False)
    assert (S == 0).all()
    _, S = run_forward(oal, c, True)
    assert torch.equal(S, c.state0)
    out = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, dstate=c.dstate)
    assert torch.equal(out[4], c.dstate)
    assert (oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY)[4] == 0).all()
    none = Case(dtype, 0, 2, 1, 5, seed=11)
    oal.oal_gated_prefill(none.Q, none.K, none.V, none.g)
    oal.oal_gated_backward(none.Q, none.K, none.V, none.g, none.dY)
    oal.oal_sync_status()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_later_tokens_change_nothing_before(oal, dtype):
    c = Case(dtype, 1, 4, 2, 500, seed=12)
    Y0, _ = run_forward(oal, c)
    for x in (c.Q, c.K, c.V):
        x[:, :, 331:] = 3.0
    c.g[:, :, 331:] = -1.0
    Y1, _ = run_forward(oal, c)
    assert torch.equal(Y0[:, :, :331], Y1[:, :, :331])


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_two_calls_of_the_same_agree_bit_for_bit(oal, dtype):
    c = Case(dtype, 2, 14, 2, 1500, seed=13)
    a, b = run_forward(oal, c, True), run_forward(oal, c, True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x, y = (oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, state0=c.state0, dstate=c.dstate) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_gradients_against_differences(oal):
    """fp32: <gradient, direction> against central differences of the oracle's
    <dY, Y> + <dstate, S_T> (64 bits, step 1e-4: error 1e-8; 1e-5 is the fp32
    gradients' own)."""
    c = Case(torch.float32, 2, 4, 2, 90, seed=14, cut=0.02, lengths=[90, 77])
    got = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=c.lengths, state0=c.state0,
                                 dstate=c.dstate)
    oal.oal_sync_status()
    gen = torch.Generator().manual_seed(5)
    base = dict(Q=c.Q, K=c.K, V=c.V, g=c.g, state0=c.state0)
    inside = c.rows(c.Q).cpu()

    def value(**kw):
        class X:
            pass
        x = X()
        x.__dict__.update(c.__dict__)
        for k, v in kw.items():
            setattr(x, k, v)
        Y, S = oracle(x, x.state0)
        return float((Y * c.dY.double().cpu() * inside).sum() + (S * c.dstate.double().cpu()).sum())

    for name, grad in zip(("Q", "K", "V", "g", "state0"), got):
        x = base[name].double()
        way = torch.randn(x.shape, generator=gen, dtype=torch.float64).cuda()
        h = 1e-4
        diff = (value(**{name: x + h * way}) - value(**{name: x - h * way})) / (2 * h)
        if name == "g":
            way = torch.where(torch.isinf(x), 0.0, way)
        mine = float((grad.double() * way).sum())
        assert abs(mine - diff) <= 1e-5 * float(grad.double().norm() * way.norm()), (name, mine, diff)


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,n", [(1, 1, 1, 1), (1, 14, 2, 4), (3, 34, 2, 7), (40, 32, 8, 64), (160, 2, 1, 160)])
def test_decode(oal, dtype, B, Hq, Hkv, n):
    c = Case(dtype, B, Hq, Hkv, 1, seed=B)
    gen = torch.Generator().manual_seed(B)
    pool = torch.randn(n, Hkv, 64, 64, generator=gen).cuda()
    slots = torch.randperm(n, generator=gen)[:B]
    c.g[0, 0, 0] = -math.inf                         # this one starts from nothing
    before = pool.clone()
    want, S = oracle(c, pool[slots.cuda()])
    y = oal.oal_gated_decode_step(c.Q[:, :, 0].contiguous(), c.K[:, :, 0].contiguous(), c.V[:, :, 0].contiguous(),
                                  c.g[:, :, 0].contiguous(), pool, SCALE, slots=slots.to(torch.int32).cuda())
    oal.oal_sync_status()
    # the state is not rounded here: bf16 only at the end
    assert rel(y, want[:, :, 0]) <= (1e-5 if dtype == torch.float32 else 2.0 ** -8)
    assert rel(pool[slots.cuda()], S) <= 1e-5
    rest = torch.ones(n, dtype=torch.bool)
    rest[slots] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])


def test_decode_spare_rows_and_bad_slots(oal):
    c = Case(torch.bfloat16, 6, 4, 2, 1, seed=20)
    args = [x[:, :, 0].contiguous() for x in (c.Q, c.K, c.V, c.g)]
    pool = torch.randn(5, 2, 64, 64, generator=torch.Generator().manual_seed(1)).cuda()
    ref = pool.clone()
    y0 = oal.oal_gated_decode_step(*[a[:2].contiguous() for a in args], ref, slots=torch.tensor([3, 1], dtype=torch.int32).cuda())
    oal.oal_sync_status()
    got = pool.clone()
    y = oal.oal_gated_decode_step(*args, got, slots=torch.tensor([3, 1, -1, -1, -1, -1], dtype=torch.int32).cuda())
    oal.oal_sync_status()                                       # -1 is no error
    assert torch.equal(y[:2], y0) and (y[2:] == 0).all() and torch.equal(got, ref)
    for bad in ([3, 1, 5, -1, -1, -1], [3, 1, -2, -1, -1, -1], [3, 1, 3, -1, 1, -1]):
        got = pool.clone()
        y = oal.oal_gated_decode_step(*args, got, slots=torch.tensor(bad, dtype=torch.int32).cuda())
        with pytest.raises(oal.OALError) as e:
            oal.oal_sync_status()
        assert e.value.status == oal.OAL_ERR_INVALID_ARG
        assert torch.equal(y[:2], y0) and (y[2:] == 0).all() and torch.equal(got, ref)


# ---------------------------------------------------------------- remap

def remapped(pool, table):
    new = pool.clone()
    for i, j in enumerate(table):
        new[i] = pool[j] if j >= 0 else 0
    return new


@pytest.mark.parametrize("n,shape,dtype", [
    (1, (4,), torch.float32), (2, (3,), torch.uint8), (7, (2, 5), torch.bfloat16), (5, (16640,), torch.float32),
    (33, (64, 64), torch.float32), (8, (2, 2145, 65), torch.float32), (700, (67,), torch.float32), (8192, (2, 2), torch.float32),
    (8192, (5,), torch.int16), (3, (1 << 21,), torch.float32), (1100, (129, 2), torch.float32)])
@pytest.mark.parametrize("kind", ["random", "cycle", "swap", "free", "fork", "stay"])
def test_remap(oal, n, shape, dtype, kind):
    gen = torch.Generator().manual_seed(n)
    pool = torch.randint(0, 200, (n,) + shape, generator=gen).to(dtype).cuda()
    table = list(range(n))
    if kind == "random":
        table = torch.randint(-1, n, (n,), generator=gen).tolist()
    elif kind == "cycle":
        table = [(i + 1) % n for i in range(n)]
    elif kind == "swap":
        table[0], table[-1] = n - 1, 0
    elif kind == "free":
        table = [-1] * n
    elif kind == "fork":
        table = [n // 2] * n
    want = remapped(pool, table)
    out = oal.oal_state_remap(pool, torch.tensor(table, dtype=torch.int32).cuda())
    oal.oal_sync_status()
    assert out is pool and torch.equal(pool, want)


def test_remap_bad_entries_stay_and_are_recorded(oal):
    pool = torch.randn(6, 40, generator=torch.Generator().manual_seed(2)).cuda()
    want = remapped(pool, [5, 1, 2, 0, -1, 5])
    oal.oal_state_remap(pool, torch.tensor([5, 6, -2, 0, -1, 5], dtype=torch.int32).cuda())
    with pytest.raises(oal.OALError) as e:
        oal.oal_sync_status()
    assert e.value.status == oal.OAL_ERR_INVALID_ARG
    assert torch.equal(pool, want)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_serving_run(oal, dtype):
    """Prompts of unequal length, a fork, decode steps on slots, an end with
    compaction, more steps: against the oracle over each sequence's own tokens."""
    B, Hq, Hkv, T, steps = 3, 4, 2, 130, 4
    lengths = [130, 50, 97]
    c = Case(dtype, B, Hq, Hkv, T, seed=30, lengths=lengths)
    pool = torch.zeros(6, Hkv, 64, 64).cuda()
    oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, SCALE, lengths=c.lengths, state=pool[:B])
    # slot 3 forks sequence 0, slot 4 forks sequence 2
    oal.oal_state_remap(pool, torch.tensor([0, 1, 2, 0, 2, -1], dtype=torch.int32).cuda())
    parents = [0, 1, 2, 0, 2]
    new = Case(dtype, 5, Hq, Hkv, 2 * steps, seed=31)
    live, ys = [0, 1, 2, 3, 4], {}
    for t in range(2 * steps):
        if t == steps:       # sequences 1 and 2 end; 3 and 4 move into their slots
            oal.oal_state_remap(pool, torch.tensor([0, 3, 4, -1, -1, -1], dtype=torch.int32).cuda())
            live = [0, 3, 4]
        rows = torch.tensor(live).cuda()
        y = oal.oal_gated_decode_step(*[x[rows, :, t].contiguous() for x in (new.Q, new.K, new.V, new.g)], pool, SCALE,
                                      slots=torch.arange(len(live), dtype=torch.int32).cuda())
        for i, s in enumerate(live):
            ys[s, t] = y[i]
    oal.oal_sync_status()
    assert (pool[3:] == 0).all()
    for s in range(5):
        p, end = parents[s], 2 * steps if s in (0, 3, 4) else steps
        n = lengths[p]
        one = Case(dtype, 1, Hq, Hkv, n + end, seed=0)
        for name in ("Q", "K", "V", "g"):
            setattr(one, name, torch.cat([getattr(c, name)[p:p + 1, :, :n], getattr(new, name)[s:s + 1, :, :end]], 2))
        want, S = oracle(one)
        got = torch.stack([ys[s, t] for t in range(end)], 1)[None]
        assert rel(got, want[:, :, n:]) <= OUT[dtype]
        if s in (0, 3, 4):
            assert rel(pool[[0, 3, 4].index(s)][None], S) <= STATE[dtype]


def test_prefix_states_of_the_quadratic_kernel_move_too(oal):
    """oal_decode_step on states that were forked and moved by a remap."""
    from grouped_quadratic_gb300 import inputs
    w = inputs.make_workload("remap", B=2, Hq=4, Hkv=2, T=70, G=3, dtype="f32", seed=77)
    Q, K, V = w.torch_inputs("cuda")
    L, group = torch.from_numpy(w.L).cuda(), torch.from_numpy(w.group).cuda()
    lay = oal.OAL_STATE_PACKED
    a, b, C = oal.oal_expand_coeffs(L, group, w.eps, lay)
    pool = torch.zeros(4, 2, oal.oal_state_rows(64, lay), 65, device="cuda")
    first = [x[:, :, :69].contiguous() for x in (Q, K, V)]
    oal.oal_prefill(*first, L, group, w.eps, a, b, C, lay, state=pool[:2])
    oal.oal_state_remap(pool, torch.tensor([1, 0, 1, -1], dtype=torch.int32).cuda())
    last = [x[:, :, 69] for x in (Q, K, V)]
    order = [1, 0, 1]
    y = oal.oal_decode_step(*[x[order].contiguous() for x in last], a, b, C, pool[:3], lay)
    Y, _ = oal.oal_prefill(Q, K, V, L, group, w.eps, a, b, C, lay)
    oal.oal_sync_status()
    assert torch.equal(y[0], y[2])
    assert rel(y, Y[order][:, :, 69]) <= 1e-5


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_prefill_in_parts(oal, dtype):
    c = Case(dtype, 2, 4, 2, 300, seed=32)
    state = torch.empty(2, 2, 64, 64, device="cuda")
    ys, at = [], 0
    for n in (1, 64, 100, 135):
        part = [x[:, :, at:at + n].contiguous() for x in (c.Q, c.K, c.V, c.g)]
        y, _ = oal.oal_gated_prefill(*part, SCALE, state=state, continue_from_state=at > 0)
        ys.append(y)
        at += n
    oal.oal_sync_status()
    want, S = oracle(c)
    assert rel(torch.cat(ys, 2), want) <= OUT[dtype] and rel(state, S) <= STATE[dtype]


def test_captured_and_replayed(oal):
    """A prefill, a backward, a decode step and a remap in one graph, replayed
    on new inputs in the same buffers."""
    c, d = Case(torch.bfloat16, 2, 4, 2, 700, seed=40), Case(torch.bfloat16, 2, 4, 2, 700, seed=41)
    q, k, v, g = (x[:, :, 0].contiguous() for x in (d.Q, d.K, d.V, d.g))
    slots, table = torch.tensor([1, 0], dtype=torch.int32).cuda(), torch.tensor([1, 0], dtype=torch.int32).cuda()

    def step(state):
        Y, _ = oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, SCALE, state=state)
        grads = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE)
        oal.oal_state_remap(state, table)
        return (Y,) + grads + (oal.oal_gated_decode_step(q, k, v, g, state, SCALE, slots=slots),)

    state = torch.empty(2, 2, 64, 64, device="cuda")
    step(state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(state)
    for src in (d, Case(torch.bfloat16, 2, 4, 2, 700, seed=42)):
        for name in ("Q", "K", "V", "g", "dY"):
            getattr(c, name).copy_(getattr(src, name))
        graph.replay()
        torch.cuda.synchronize()
        again = torch.empty_like(state)
        want = step(again)
        oal.oal_sync_status()
        assert all(torch.equal(x, y) for x, y in zip(out, want)) and torch.equal(state, again)


def test_on_another_stream(oal):
    c = Case(torch.bfloat16, 2, 14, 2, 3000, seed=43)
    want = run_forward(oal, c, True)
    grads = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, state0=c.state0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(3):
        got.append(run_forward(oal, c, True, stream=side))
        more = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, state0=c.state0, stream=side)
        torch.full((1 << 22,), math.nan, device="cuda")     # would land in scratch that was freed too early
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(grads, more))
    oal.oal_sync_status()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))


def test_offsets_beyond_32_bits(oal):
    """More than 2^32 bytes and 2^31 elements of Q and Y: the last rows against
    a call on the last part alone that goes on from the state before it."""
    T, Hq, tail = 1 << 20, 36, 1000
    gen = torch.Generator(device="cuda").manual_seed(3)
    Q = torch.randn(1, Hq, T, 64, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert Q.numel() > 1 << 31
    K, V = (torch.randn(1, 1, T, 64, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = torch.full((1, 1, T), -0.01, device="cuda")
    Y, S = oal.oal_gated_prefill(Q, K, V, g)
    cut = lambda a, b: [x[:, :, a:b].contiguous() for x in (Q, K, V, g)]
    _, S0 = oal.oal_gated_prefill(*cut(T - tail - 4000, T - tail))       # exp(-40) of what is before
    y, s = oal.oal_gated_prefill(*cut(T - tail, T), state=S0, continue_from_state=True)
    oal.oal_sync_status()
    assert rel(Y[:, :, T - tail:], y) <= OUT[torch.bfloat16]
    assert rel(S, s) <= STATE[torch.bfloat16]


def test_outputs_made_in_a_call_on_another_stream(oal):
    """The current stream is busy when the call makes its outputs (zeroed there,
    as there are lengths): the kernels on the other stream come behind that."""
    c = Case(torch.bfloat16, 2, 14, 2, 3000, seed=44, lengths=[3000, 1701])
    grads = lambda **kw: oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, lengths=c.lengths, state0=c.state0, **kw)
    want = oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, lengths=c.lengths) + grads()
    work = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    work @ work
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):                       # about 5 ms
        work @ work
    got = oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, lengths=c.lengths, stream=side) + grads(stream=side)
    torch.cuda.synchronize()
    oal.oal_sync_status()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# Constant gates whose decay over a chunk (the first two; over a token: the
# third) lies nearly half way between two fp32 numbers: a decay carried as one
# fp32 factor is off by the same 2^-25 every time, 3e-5 to 1e-4 of the state
# after these many chunks.  Independent roundings are what the tolerances
# count: 4096 chunks of 64 tokens, sqrt(4160) 2^-24 = 4e-6.
SLOW = [-8.181881980817707e-07, -2.6682809561862086e-07, -1e-5, -3e-6]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", SLOW)
@pytest.mark.parametrize("T", [65536, 262143])
def test_slow_gates_over_many_chunks(oal, dtype, gate, T):
    gen = torch.Generator(device="cuda").manual_seed(50)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    Q, K, V, dY = (n(1, 1, T, 64).to(dtype) for _ in range(4))
    state0, dstate = n(1, 1, 64, 64), n(1, 1, 64, 64)
    g = torch.full((1, 1, T), gate, device="cuda")
    # S_T = sum_t e^{(T-1-t) g} k_t v_t^T + e^{T g} S_0, and its like for the gradient
    age = torch.arange(T, device="cuda", dtype=torch.float64) * float(g[0, 0, 0])
    last = math.exp(T * float(g[0, 0, 0]))
    S = (K[0, 0].double() * age.flip(0).exp()[:, None]).T @ V[0, 0].double() + last * state0[0, 0].double()
    first = math.exp(float(g[0, 0, 0]))
    R = SCALE * first * (Q[0, 0].double() * age.exp()[:, None]).T @ dY[0, 0].double() + last * dstate[0, 0].double()
    _, state = oal.oal_gated_prefill(Q, K, V, g, SCALE, state=state0.clone(), continue_from_state=True)
    grads = oal.oal_gated_backward(Q, K, V, g, dY, SCALE, state0=state0, dstate=dstate)
    oal.oal_sync_status()
    assert rel(state[0, 0], S) <= STATE[dtype]
    assert rel(grads[4][0, 0], R) <= STATE[dtype]


@pytest.mark.parametrize("gate", [-8.9e-8, -2.6682809561862086e-07, -1e-5])
def test_slow_gates_over_many_steps(oal, gate):
    """16384 decode steps: sqrt(16384) 2^-24 = 8e-6 from roundings that are
    independent; half a step each time the same way would be 16384 2^-25 = 5e-4."""
    steps = 16384
    gen = torch.Generator(device="cuda").manual_seed(51)
    q, k, v = (torch.randn(steps, 1, 1, 64, generator=gen, device="cuda") for _ in range(3))
    state0 = torch.randn(1, 1, 64, 64, generator=gen, device="cuda")
    g = torch.full((1, 1), gate, device="cuda")
    state, y = state0.clone(), torch.empty(1, 1, 64, device="cuda")
    for t in range(steps):
        oal.oal_gated_decode_step(q[t], k[t], v[t], g, state, SCALE, y=y)
    oal.oal_sync_status()
    age = torch.arange(steps, device="cuda", dtype=torch.float64) * float(g)
    S = (k[:, 0, 0].double() * age.flip(0).exp()[:, None]).T @ v[:, 0, 0].double() + math.exp(steps * float(g)) * state0[0, 0].double()
    assert rel(state[0, 0], S) <= 1e-5


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,T,at", [
    (1, 2, 1, 1, 0), (2, 3, 1, 130, 0), (1, 4, 2, 200, 70), (1, 2, 2, 5000, 3001), (160, 3, 3, 170, 100),
    (1, 1, 1, 20000, 64)])
def test_a_cut_shuts_out_a_state_that_is_not_finite(oal, dtype, bad, B, Hq, Hkv, T, at):
    """Behind a cut gate a state starts from nothing, whatever was in it; the
    gradient of the state does so in front of one."""
    c = Case(dtype, B, Hq, Hkv, T, seed=60)
    c.g[:, :, at] = -math.inf
    c.g[:, :, 130::400] = -80.0                      # (chunks of every kind of gates behind it)
    dirty = torch.full_like(c.state0, bad)
    Y0, S0 = run_forward(oal, c, True)
    G0 = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, state0=c.state0, dstate=c.dstate)
    clean = c.state0
    c.state0 = dirty
    Y1, S1 = run_forward(oal, c, True)
    G1 = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, state0=dirty, dstate=c.dstate)
    G2 = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, state0=clean, dstate=dirty)
    oal.oal_sync_status()
    assert torch.equal(S0, S1) and torch.equal(Y0[:, :, at:], Y1[:, :, at:])
    assert torch.equal(G0[0][:, :, at:], G1[0][:, :, at:])                        # dQ behind the cut
    assert torch.equal(G0[3][:, :, at:], G1[3][:, :, at:])                        # dg
    for i in (1, 2, 4):                              # dK, dV and dstate0 do not see the state
        assert torch.equal(G0[i], G1[i])
    assert torch.equal(G0[0], G2[0])                                             # dQ does not see its gradient
    for i in (1, 2, 3):
        assert torch.equal(G0[i][:, :, :at], G2[i][:, :, :at])
    assert torch.equal(G0[4], G2[4])


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_decode_cut_shuts_out_a_state_that_is_not_finite(oal, dtype):
    c = Case(dtype, 3, 4, 2, 1, seed=61)
    c.g[:] = torch.tensor([-math.inf, -104.0, -1e30]).cuda()[:, None, None]
    args = [x[:, :, 0].contiguous() for x in (c.Q, c.K, c.V, c.g)]
    want = oal.oal_gated_decode_step(*args, c.state0, SCALE)
    for bad in (math.nan, math.inf, -math.inf):
        state = torch.full_like(c.state0, bad)
        assert torch.equal(oal.oal_gated_decode_step(*args, state, SCALE), want)
        assert torch.equal(state, c.state0)
    oal.oal_sync_status()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [-1.8, -0.9, -0.3])
def test_only_far_keys(oal, dtype, gate):
    """Rows that see nothing but the last keys of the chunk's other half."""
    c = Case(dtype, 1, 2, 1, 64, seed=71)
    c.g = torch.full_like(c.g, gate)
    c.K[:, :, :24] = 0
    c.K[:, :, 32:] = 0
    check_forward(oal, c, False)
    Y, _ = run_forward(oal, c)
    want, _ = oracle(c)
    for t in range(64):                      # row by row: the first ones are 1e40 times the last
        err, size = (float(x.norm()) for x in (Y[:, :, t].double().cpu() - want[:, :, t], want[:, :, t]))
        if size > 1e-30:
            assert err <= OUT[dtype] * size, t
    got = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE)
    oal.oal_sync_status()
    grads = oracle(c, backward=True)
    for t in range(64):
        err, size = (float(x.norm()) for x in (got[0][:, :, t].double().cpu() - grads[0][:, :, t], grads[0][:, :, t]))
        if size > 1e-30:
            assert err <= OUT[dtype] * size, t


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-8, 1e4, 1e8])
@pytest.mark.parametrize("gate", [-1.8, -0.9, -0.4, -0.16, -0.01])
def test_large_and_small_inputs(oal, dtype, size, gate):
    """Results of up to 1e27 (and down to 1e-24) are inside the types' range,
    whatever the gates: no factor on the way may leave it."""
    c = Case(dtype, 1, 3, 1, 150, seed=70)
    c.g = torch.full_like(c.g, gate)
    c.g[:, :, 77] = -math.inf
    for name, f in (("Q", size), ("K", size), ("V", size), ("state0", size * size)):
        setattr(c, name, (getattr(c, name) * f).contiguous())
    check_forward(oal, c, True)
    check_backward(oal, c, True)


def test_large_inputs_in_some_segments(oal):
    """bf16, segments of three chunks, some of which outgrow the first way of
    forming them: all come out as by themselves."""
    c = Case(torch.bfloat16, 160, 9, 3, 170, seed=72, lengths=[170, 169, 128, 129, 5, 0, 64, 65] * 20)
    c.g = torch.full_like(c.g, -0.9)
    Y0, S0 = run_forward(oal, c, True)
    for name, f in (("Q", 1e8), ("K", 1e8), ("V", 1e8), ("state0", 1e16)):
        x = getattr(c, name)
        x[::3] *= f
    Y1, S1 = run_forward(oal, c, True)
    small = torch.arange(160, device="cuda") % 3 != 0
    assert torch.equal(Y0[small], Y1[small]) and torch.equal(S0[small], S1[small])
    check_forward(oal, c, True)
    for b in (0, 3, 6, 9):                   # by themselves, as the large ones hide the others in a norm
        one = Case(torch.bfloat16, 1, 9, 3, 170, seed=72, lengths=[int(c.lengths[b])])
        for name in ("Q", "K", "V", "g", "state0"):
            setattr(one, name, getattr(c, name)[b:b + 1].clone())
        check_forward(oal, one, True)


# ---------------------------------------------------------------- row by row

def rows_off(got, want, inside=None):
    """The largest error of a row (of the last dimension), relative to the row's
    norm or the tensor's root mean square of them, whichever is larger: the
    roundings that a tensor's tolerance counts are those of the row's own terms,
    which may cancel, but are of the size of other rows' terms."""
    got, want = got.double().cpu(), want.double().cpu()
    err, size = (got - want).norm(dim=-1), want.norm(dim=-1)
    if inside is not None:
        inside = inside[..., 0].cpu()
        err, size = err[inside], size[inside]
    assert torch.isfinite(err).all()
    rms = float(size.square().mean().sqrt())
    return float((err / size.clamp(min=max(rms, 1e-30))).max()) if err.numel() else 0.0


def every_kind_of_gate(c):
    """Chunk after chunk as drawn, four times, thirty times as steep, and with a cut."""
    for i, t0 in enumerate(range(0, c.T, 64)):
        c.g[:, :, t0:t0 + 64] *= (1.0, 30.0, 4.0, 1.0)[i % 4]
        if i % 4 == 3:
            c.g[:, :, t0 + i % 64] = -math.inf
    return c


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,T,span,lengths", [
    (2, 10, 2, 191, 30.0, [191, 17]), (1, 7, 1, 1000, 30.0, None), (3, 9, 1, 257, 3.0, [257, 256, 3]),
    # several chunks a segment of the prefill and a block of the backward
    (160, 3, 3, 170, 3.0, [170, 169, 128, 129, 5, 0, 64, 65] * 20), (60, 10, 2, 400, 3.0, None),
    (100, 5, 5, 330, 30.0, list(range(231, 331))),
    # many segments of few states, some sequences shorter; more than the split scan's round of 256
    (3, 4, 2, 3000, 300.0, [3000, 0, 1101]), (2, 1, 1, 17000, 2000.0, [17000, 16383])])
def test_row_by_row(oal, dtype, B, Hq, Hkv, T, span, lengths):
    c = every_kind_of_gate(Case(dtype, B, Hq, Hkv, T, seed=80 + B, span=span, lengths=lengths))
    Y, state = run_forward(oal, c, True)
    want, S = oracle(c, c.state0)
    assert rows_off(Y, want, c.rows(Y)) <= OUT[dtype]
    assert rows_off(state.flatten(2), S.flatten(2)) <= STATE[dtype]
    got = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, lengths=c.lengths, state0=c.state0, dstate=c.dstate)
    oal.oal_sync_status()
    want = oracle(c, c.state0, c.dstate, backward=True)
    for name, x, w in zip(("dQ", "dK", "dV"), got, want):
        assert rows_off(x, w, c.rows(x)) <= OUT[dtype], name
    assert rows_off(got[3], want[3]) <= DG[dtype]                       # (a row: a sequence and head)
    assert rows_off(got[4].flatten(2), want[4].flatten(2)) <= STATE[dtype]


@pytest.mark.parametrize("span", [30.0, 300.0, 2000.0])
def test_gate_gradients_as_sums_of_fp32_products(oal, span):
    """dg of bf16 inputs: products of states in all of their bits.  A sum takes
    at most 12 steps in the tensor cores, which cut: 12 * 2^-23 = 1.4e-6; the
    sums over a chunk's tokens behind that add sqrt(128) 2^-24 = 7e-7."""
    c = Case(torch.bfloat16, 1, 4, 1, 4096, seed=90, span=span)
    got = oal.oal_gated_backward(c.Q, c.K, c.V, c.g, c.dY, SCALE, state0=c.state0, dstate=c.dstate)
    oal.oal_sync_status()
    want = oracle(c, c.state0, c.dstate, backward=True)
    assert rel(got[3], want[3]) <= 2.1e-6


# ---------------------------------------------------------------- next to other calls

def test_the_quadratic_kernel_reads_what_a_gated_call_just_wrote(oal):
    """Y of a gated prefill as Q, K and V of oal_prefill with nothing between
    the two calls, whose kernels overlap at their ends."""
    from grouped_quadratic_gb300 import inputs
    B, H, T = 2, 8, 2000
    w = inputs.make_workload("chain", B=1, Hq=H, Hkv=H, T=16, G=3, dtype="bf16", seed=78)
    L, group = torch.from_numpy(w.L).cuda(), torch.from_numpy(w.group).cuda()
    lay = oal.OAL_STATE_PACKED
    a, b, C = oal.oal_expand_coeffs(L, group, w.eps, lay)
    c = Case(torch.bfloat16, B, H, H, T, seed=95)
    Y, state = torch.empty_like(c.Q), torch.empty_like(c.state0)
    Z, prefix = torch.empty_like(c.Q), torch.empty(B, H, oal.oal_state_rows(64, lay), 65, device="cuda")
    gws = torch.empty(oal.oal_gated_prefill_workspace_bytes(B, H, H, T), dtype=torch.uint8, device="cuda")
    ows = torch.empty(oal.oal_prefill_workspace_bytes(B, H, H, T, layout=lay), dtype=torch.uint8, device="cuda")

    def gated():
        oal.oal_gated_prefill(c.Q, c.K, c.V, c.g, SCALE, state=state, Y=Y, workspace=gws)

    def quadratic():
        oal.oal_prefill(Y, Y, Y, L, group, w.eps, a, b, C, lay, state=prefix, Y=Z, workspace=ows)

    gated()
    torch.cuda.synchronize()
    quadratic()
    oal.oal_sync_status()
    want = Z.clone(), prefix.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gated()
        quadratic()
    for run in [lambda: (gated(), quadratic())] * 3 + [graph.replay] * 3:
        for x in (Y, Z, prefix):
            x.zero_()
        torch.cuda.synchronize()
        run()
        oal.oal_sync_status()
        assert torch.equal(Z, want[0]) and torch.equal(prefix, want[1])


def test_calls_at_once_on_two_streams(oal):
    """Prefills and backwards that share the SMs, a workspace each."""
    c, d = Case(torch.bfloat16, 4, 8, 4, 3000, seed=96), Case(torch.bfloat16, 3, 6, 2, 2500, seed=97, lengths=[2500, 700, 1])
    forward = lambda x, **kw: oal.oal_gated_prefill(x.Q, x.K, x.V, x.g, SCALE, lengths=x.lengths, **kw)
    back = lambda x, **kw: oal.oal_gated_backward(x.Q, x.K, x.V, x.g, x.dY, SCALE, lengths=x.lengths, state0=x.state0, **kw)
    want = forward(c) + back(c), forward(d) + back(d)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(4):
        for out, x, stream in ((got[0], c, one), (got[1], d, two)):
            with torch.cuda.stream(stream):
                out.append(forward(x) + back(x))
    torch.cuda.synchronize()
    oal.oal_sync_status()
    for outs, ref in zip(got, want):
        for out in outs:
            assert all(torch.equal(x, y) for x, y in zip(out, ref))
