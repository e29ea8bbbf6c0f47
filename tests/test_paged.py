"""Rotary positions, the paged cache and its attention: the host's plan, and what
is refused before any launch (no GPU needed).  Results: test_paged_gpu.py."""
import ctypes
import math

import pytest
import torch

P = ctypes.c_void_p(4096)      # a fake, aligned address; never dereferenced
NULL, ODD = ctypes.c_void_p(0), ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    return oal.load_library()


def strides(*x):
    return (ctypes.c_int64 * len(x))(*x)


def rope(lib, **kw):
    a = dict(Q=P, K=P, dtype=1, strides=None, B=2, Hq=4, Hkv=2, T=100, d=64, plan=P, form=0, positions=None,
             n_axes=0, past=None, lengths=None, inverse=0, Yq=P, Yk=P, stream=None)
    a.update(kw)
    return lib.oal_rope(*a.values())


def append(lib, **kw):
    a = dict(Q=P, K=P, V=P, dtype=1, strides=None, B=2, Hq=4, Hkv=2, T=100, d=64, dv=64, plan=P, form=0,
             positions=None, n_axes=0, past=P, lengths=None, Kp=P, Vp=P, n_pages=8, page_size=16,
             page_stride=2 * 16 * 64, table=P, max_pages=10, Yq=P, stream=None)
    a.update(kw)
    return lib.oal_page_append(*a.values())


def attend(lib, **kw):
    a = dict(Q=P, dtype=1, B=2, Hq=4, Hkv=2, T=100, d=64, dv=64, Kp=P, Vp=P, n_pages=8, page_size=16,
             page_stride=2 * 16 * 64, table=P, max_pages=10, past=P, lengths=None, scale=0.125, cap=0.0, window=0,
             slopes=None, prefix=None, first=None, Y=P, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.oal_paged_attention(*a.values())


TURNS = [(dict(d=128), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(dtype=2), 1),
         (dict(form=2), 1), (dict(B=1 << 20, T=1 << 20), 2), (dict(Hq=1 << 17), 2), (dict(positions=P), 1),
         (dict(positions=ODD, n_axes=1), 1), (dict(past=ODD), 1), (dict(lengths=ODD), 1), (dict(plan=ODD), 1),
         (dict(Q=ODD), 1), (dict(K=ODD), 1), (dict(Yq=NULL), 1)]


@pytest.mark.parametrize("kw,status", TURNS + [
    (dict(Q=NULL), 1), (dict(Yk=NULL), 1), (dict(plan=NULL), 1),
    (dict(strides=strides(64, 64, 60, 64, 64, 64)), 1), (dict(strides=strides(64, 64, 64, 64, -64, 64)), 1)])
def test_rope_refuses(lib, kw, status):
    assert rope(lib, **kw) == status
    assert lib.oal_last_error().decode()


PAGES = [(dict(n_pages=-1), 1), (dict(max_pages=-1), 1), (dict(page_size=0), 1), (dict(page_size=48), 1),
         (dict(page_size=8), 2), (dict(page_size=1 << 17, page_stride=1 << 30), 2), (dict(max_pages=1 << 27), 2),
         (dict(page_stride=2 * 16 * 64 - 8), 1), (dict(page_stride=2 * 16 * 64 + 4), 1), (dict(Kp=NULL), 1),
         (dict(Vp=ODD), 1), (dict(table=NULL), 1), (dict(past=NULL), 1)]


@pytest.mark.parametrize("kw,status", TURNS + PAGES + [
    (dict(dv=32), 2), (dict(K=NULL), 1), (dict(V=NULL), 1), (dict(plan=NULL), 1),
    (dict(strides=strides(64, 64, 64, 64, 64, 64, 64, 64, 62)), 1)])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status
    assert lib.oal_last_error().decode()


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(d=128), 2), (dict(dv=32), 2), (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(B=-1), 1), (dict(T=-1), 1),
    (dict(dtype=3), 1), (dict(Hq=258), 2), (dict(B=40000), 2), (dict(T=1 << 28), 2), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(cap=-1.0), 1),
    (dict(cap=math.nan), 1), (dict(cap=1e-40), 1), (dict(B=1 << 13, T=1 << 19), 2), (dict(cap=math.inf), 1), (dict(window=-1), 1), (dict(Q=NULL), 1), (dict(Y=ODD), 1),
    (dict(lengths=ODD), 1), (dict(slopes=ODD), 1), (dict(prefix=ODD), 1), (dict(first=ODD), 1), (dict(ws=NULL, T=1, max_pages=1 << 16), 1),
    (dict(ws=ctypes.c_void_p(4096 + 16)), 1), (dict(ws_bytes=100), 1),
    (dict(T=1, max_pages=1 << 16, ws_bytes=1024), 1)])
def test_attention_refuses(lib, kw, status):
    assert attend(lib, **kw) == status
    assert lib.oal_last_error().decode()


def test_nothing_to_do(lib):
    for kw in (dict(B=0), dict(T=0)):
        assert rope(lib, Q=NULL, K=NULL, plan=NULL, **kw) in (0, 1)
        assert rope(lib, **kw) == append(lib, **kw) == attend(lib, **kw) == 0
    assert lib.oal_last_call_launches() == 0


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,Hq,Hkv,T", [(1, 14, 2, 1), (64, 32, 8, 1), (1, 8, 8, 333), (2, 14, 2, 2048), (1, 128, 1, 3)])
@pytest.mark.parametrize("page,most", [(16, 1), (16, 5), (64, 128), (128, 4096)])
def test_workspace_holds_whatever_the_window(lib, dtype, B, Hq, Hkv, T, page, most):
    need = lib.oal_paged_attention_workspace_bytes(B, Hq, Hkv, T, 64, 64, dtype, page, most)
    assert need >= 256
    size = dict(B=B, Hq=Hq, Hkv=Hkv, T=T, dtype=dtype, page_size=page, page_stride=Hkv * page * 64, max_pages=most)
    # one byte less is refused, whatever the window
    for window in (0, 1, 100, 1000):
        assert attend(lib, window=window, ws_bytes=need - 1, **size) == 1


def test_workspace_of_sizes_that_are_refused(lib):
    f = lib.oal_paged_attention_workspace_bytes
    assert f(1, 5, 2, 1, 64, 64, 1, 16, 4) == 0 and f(1, 4, 2, 1, 32, 64, 1, 16, 4) == 0
    assert f(1, 4, 2, 1, 64, 64, 1, 24, 4) == 0 and f(0, 4, 2, 1, 64, 64, 1, 16, 4) == 256


@pytest.mark.parametrize("base", [1e4, 5e5, 1e6])
def test_plan_against_exact_turns(lib, base):
    """turns = freq / 2 pi modulo 1 in units of 2^-64, within what freq / 2 pi in two doubles gives (2^-60)."""
    from decimal import Decimal, getcontext
    from grouped_quadratic_gb300 import oal
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    freq = [base ** (-r / 32) for r in range(32)]
    freq[5], freq[6], freq[7] = 0.0, -freq[6], 1234.5
    plan = oal.oal_rope_plan(freq, list(range(32)), device="cpu")
    assert plan.shape == (2, 32) and plan[1].tolist() == list(range(32))
    for f, got in zip(freq, plan[0].tolist()):
        turns = Decimal(f) / two_pi
        turns -= turns.to_integral_value(rounding="ROUND_FLOOR")
        off = (Decimal(got % 2 ** 64) - turns * 2 ** 64) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # 2^-105 of a value of up to 197 turns, the truncation to 2^-64, and its rounding to even numbers
        assert off <= 4, (f, off)


def test_plan_refuses(lib):
    from grouped_quadratic_gb300 import oal
    with pytest.raises(oal.OALError):
        oal.oal_rope_plan([math.nan] * 32, device="cpu")
    with pytest.raises(oal.OALError):
        oal.oal_rope_plan([1.0] * 31, device="cpu")
    with pytest.raises(oal.OALError):
        oal.oal_rope_plan([1.0] * 32, [-1] * 32, device="cpu")
    assert lib.oal_rope_plan(None, None, None) == 1


def test_binding_refuses_host_tensors_and_shapes(lib):
    from grouped_quadratic_gb300 import oal
    q, k = torch.zeros(1, 4, 3, 64), torch.zeros(1, 2, 3, 64)
    plan = torch.zeros(2, 32, dtype=torch.int64)
    pool, table, past = torch.zeros(4, 2, 16, 64), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: oal.oal_rope(q, k, plan), lambda: oal.oal_rope(q, k, None), lambda: oal.oal_rope(q[0], k, plan),
                 lambda: oal.oal_rope(q, k.transpose(2, 3).contiguous().transpose(2, 3), plan),
                 lambda: oal.oal_rope(q, k, plan, positions=torch.zeros(3, 1, 4, dtype=torch.int32)),
                 lambda: oal.oal_page_append(q, k, k, plan, pool, pool, table, past),
                 lambda: oal.oal_page_append(q, k, k, plan, pool, pool, table, None),
                 lambda: oal.oal_page_append(q, k, k[:, :1], plan, pool, pool, table, past),
                 lambda: oal.oal_page_append(q, k, k, plan, pool[:, :1], pool[:, :1], table, past),
                 lambda: oal.oal_page_append(None, k, k, plan, pool, pool, table, past, Yq=q),
                 lambda: oal.oal_paged_attention(q, pool, pool, table, past),
                 lambda: oal.oal_paged_attention(q, pool, pool[:, :, ::2], table, past),
                 lambda: oal.oal_paged_attention(q, pool, pool.to(torch.bfloat16), table, past),
                 lambda: oal.oal_paged_attention(q, pool, pool, table, past, slopes=torch.zeros(2)),
                 lambda: oal.oal_paged_attention(q, pool, pool, table, past, first=torch.zeros(1, 4, dtype=torch.int32))):
        with pytest.raises(oal.OALError):
            call()
