"""C-ABI checks that need no GPU: the library builds, loads, exports every
symbol include/oal.h declares, and rejects bad arguments on the host."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "oal.h")


@pytest.fixture(scope="module")
def lib():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    return oal.load_library()


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(oal_[a-z0-9_]+)\s*\(",
                       text, flags=re.M)
    return sorted(set(names))


def test_header_declares_the_boundary():
    names = declared_functions()
    for required in ["oal_expand_coeffs", "oal_prefill", "oal_prefill_workspace_bytes",
                     "oal_decode_step", "oal_decode_workspace_bytes", "oal_state_rows",
                     "oal_state_elems", "oal_sync_status", "oal_last_error"]:
        assert required in names


def test_library_exports_every_declared_symbol(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name


def test_state_sizes(lib):
    from grouped_quadratic_gb300 import oal
    assert oal.oal_state_rows(64, oal.OAL_STATE_FULL) == 4161
    assert oal.oal_state_rows(64, oal.OAL_STATE_PACKED) == 2145
    assert oal.oal_state_elems(64, 64, oal.OAL_STATE_FULL) * 4 == 1081860
    assert oal.oal_state_elems(64, 64, oal.OAL_STATE_PACKED) * 4 == 557700
    assert oal.oal_coeff_table_elems(64, oal.OAL_STATE_PACKED) == 2080
    assert oal.oal_state_rows(64, 7) == 0
    assert oal.oal_version()


def _prefill_raw(lib, **kw):
    from grouped_quadratic_gb300 import oal
    p = ctypes.c_void_p(4096)  # a fake, aligned address; never dereferenced
    args = dict(Q=p, K=p, V=p, dtype=oal.OAL_BF16, B=1, Hq=4, Hkv=2, T=8, d=64, dv=64,
                L=p, group=p, G=3, eps=1e-6, a=p, b=p, C=p, layout=oal.OAL_STATE_FULL,
                state=p, cont=0, Y=p, chunk=0, ws=p, ws_bytes=0, stream=None)
    args.update(kw)
    return lib.oal_prefill(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), 2), (dict(dv=128), 2), (dict(G=0), 2), (dict(G=8), 2),
    (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(dtype=7), 1), (dict(layout=3), 1),
    (dict(chunk=96), 1), (dict(eps=0.0), 1), (dict(T=-1), 1),
    (dict(Q=ctypes.c_void_p(0)), 1), (dict(K=ctypes.c_void_p(4100)), 1),
    (dict(ws_bytes=16), 1),
])
def test_prefill_rejects_bad_arguments_on_host(lib, kw, status):
    assert _prefill_raw(lib, **kw) == status
    assert lib.oal_last_error().decode() != ""


def _contrib_raw(lib, **kw):
    from grouped_quadratic_gb300 import oal
    p = ctypes.c_void_p(4096)  # a fake, aligned address; never dereferenced
    args = dict(Q=p, K=p, dtype=oal.OAL_BF16, P=2, Hq=4, Hkv=2, T=8, d=64, lengths=None,
                chi=p, ws=p, ws_bytes=1 << 20, stream=None)
    args.update(kw)
    return lib.oal_contribution_scores(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), 2), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(dtype=5), 1), (dict(P=-1), 1),
    (dict(T=-2), 1), (dict(chi=ctypes.c_void_p(0)), 1), (dict(Q=ctypes.c_void_p(4100)), 1),
    (dict(lengths=ctypes.c_void_p(4098)), 1), (dict(ws=ctypes.c_void_p(4096 + 16)), 1),
    (dict(ws_bytes=8), 1),
])
def test_contribution_scores_reject_bad_arguments_on_host(lib, kw, status):
    assert _contrib_raw(lib, **kw) == status
    assert lib.oal_last_error().decode() != ""


def test_workspace_queries(lib):
    from grouped_quadratic_gb300 import oal
    n = oal.oal_prefill_workspace_bytes(1, 14, 2, 4096, layout=oal.OAL_STATE_PACKED)
    assert n > 0
    assert oal.oal_prefill_workspace_bytes(1, 14, 2, 4096, chunk=96) == 0
    assert oal.oal_decode_workspace_bytes(64, 14, 2) > 0
    n = oal.oal_contribution_workspace_bytes(40, 14, 2, 4096)
    assert n == 40 * 32 * 64 * 4 * (2 + 2 * 14)
    assert oal.oal_contribution_workspace_bytes(40, 14, 2, 4096, d=32) == 0


def test_intra_heads_hook_validates_on_host(lib):
    # the test hook for the intra-chunk kernel's block shape takes 0, 1 or 2
    for bad in (-1, 3):
        assert lib.oal_debug_intra_heads(bad) == 1   # OAL_ERR_INVALID_ARG
    for good in (1, 2, 0):
        assert lib.oal_debug_intra_heads(good) == 0


def test_missing_library_fails_loudly(tmp_path):
    from grouped_quadratic_gb300 import oal
    saved = oal._lib
    oal._lib = None
    try:
        with pytest.raises(oal.OALError):
            oal.load_library(str(tmp_path / "nope.so"))
    finally:
        oal._lib = saved


def test_calls_order_what_they_make_before_their_stream(monkeypatch):
    """oal_prefill, its backward, the decode step, the scores and the tables on a
    stream that is not the current one: the stream waits for the current one,
    from whose pool they allocate, and keeps their memory."""
    import torch
    from grouped_quadratic_gb300 import oal

    class Stream:
        device, cuda_stream = torch.device("cuda", 0), 77

        def __init__(self):
            self.calls = []

        def wait_stream(self, other):
            self.calls.append(("wait", other))

    class Lib:                                    # sizes, and calls that succeed
        def __getattr__(self, name):
            return lambda *a: 64 if name.endswith(("_bytes", "_elems", "_rows")) else 0

    now, side = Stream(), Stream()
    monkeypatch.setattr(oal, "load_library", lambda: Lib())
    monkeypatch.setattr(oal, "_need_cuda", lambda *t: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: s.calls.append(("record", t)))
    z = torch.zeros
    Q, K, L, g = z(1, 2, 8, 64), z(1, 1, 8, 64), z(2, 3, 3), z(2, 64, dtype=torch.int32)
    calls = [lambda: oal.oal_expand_coeffs(L, g, 0.1, stream=side),
             lambda: oal.oal_prefill(Q, K, K, L, g, 0.1, L, L, L, stream=side),
             lambda: oal.oal_prefill_backward(Q, K, K, Q, L, g, 0.1, stream=side),
             lambda: oal.oal_decode_step(Q[:, :, 0], K[:, :, 0], K[:, :, 0], L, L, L, K, stream=side),
             lambda: oal.oal_contribution_scores(Q, K, stream=side)]
    for call, made in zip(calls, (3, 3, 5, 2, 2)):
        side.calls.clear()
        call()
        assert side.calls[0] == ("wait", now) and len(side.calls) == 1 + made
    assert now.calls == []
