"""Gated recurrence and state remap: what is refused on the host, before any
launch (no GPU needed).  Results are compared in test_gated_gpu.py."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(4096)      # a fake, aligned address; never dereferenced
NULL, ODD = ctypes.c_void_p(0), ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    return oal.load_library()


def prefill(lib, **kw):
    a = dict(Q=P, K=P, V=P, dtype=1, g=P, B=2, Hq=4, Hkv=2, T=4096, d=64, dv=64, scale=0.125,
             lengths=None, state=P, cont=0, Y=P, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.oal_gated_prefill(*a.values())


def backward(lib, **kw):
    a = dict(Q=P, K=P, V=P, dtype=1, g=P, dY=P, B=2, Hq=4, Hkv=2, T=4096, d=64, dv=64, scale=0.125,
             lengths=None, state0=None, dstate=None, dQ=P, dK=P, dV=P, dg=P, dstate0=None, ws=P,
             ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.oal_gated_backward(*a.values())


def decode(lib, **kw):
    a = dict(q=P, k=P, v=P, dtype=1, g=P, B=2, Hq=4, Hkv=2, d=64, dv=64, scale=0.125, slots=None,
             n_slots=2, state=P, y=P, stream=None)
    a.update(kw)
    return lib.oal_gated_decode_step(*a.values())


SIZES = [(dict(d=128), 2), (dict(dv=32), 2), (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(B=-1), 1),
         (dict(dtype=3), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(T=-1), 1), (dict(T=(1 << 30) + 1), 2), (dict(B=1 << 20, T=1 << 20), 2),
    (dict(Q=NULL), 1), (dict(K=NULL), 1), (dict(V=ODD), 1), (dict(g=NULL), 1), (dict(Y=NULL), 1),
    (dict(state=NULL), 1), (dict(lengths=ODD), 1), (dict(ws=NULL), 1),
    (dict(ws=ctypes.c_void_p(4096 + 16)), 1), (dict(ws_bytes=1024), 1)])
def test_prefill_refuses(lib, kw, status):
    assert prefill(lib, **kw) == status
    assert lib.oal_last_error().decode()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(T=-3), 1), (dict(Q=NULL), 1), (dict(dY=NULL), 1), (dict(dQ=ODD), 1), (dict(dK=NULL), 1),
    (dict(dV=NULL), 1), (dict(dg=NULL), 1), (dict(state0=ODD), 1), (dict(dstate=ODD), 1),
    (dict(dstate0=ODD), 1), (dict(lengths=ODD), 1), (dict(ws=NULL), 1), (dict(ws_bytes=1024), 1)])
def test_backward_refuses(lib, kw, status):
    assert backward(lib, **kw) == status
    assert lib.oal_last_error().decode()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(n_slots=1), 1), (dict(n_slots=-1), 1), (dict(q=NULL), 1), (dict(k=ODD), 1), (dict(g=NULL), 1),
    (dict(y=NULL), 1), (dict(state=NULL), 1), (dict(slots=ODD), 1)])
def test_decode_refuses(lib, kw, status):
    assert decode(lib, **kw) == status
    assert lib.oal_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(n=8193), 2), (dict(pool=NULL), 1), (dict(pool=ODD), 1), (dict(map=NULL), 1),
    (dict(bytes=1 << 45), 2)])
def test_remap_refuses(lib, kw, status):
    a = dict(pool=P, bytes=1024, n=4, map=P, stream=None)
    a.update(kw)
    assert lib.oal_state_remap(*a.values()) == status
    assert lib.oal_last_error().decode()


def test_empty_calls_launch_nothing(lib):
    assert prefill(lib, B=0) == 0
    assert backward(lib, B=0) == 0
    assert backward(lib, T=0) == 0                 # no dstate0: nothing to write
    assert decode(lib, B=0, n_slots=0) == 0
    assert lib.oal_state_remap(NULL, 64, 0, NULL, None) == 0
    assert lib.oal_state_remap(P, 0, 3, P, None) == 0


def test_workspace_sizes(lib):
    from grouped_quadratic_gb300 import oal
    assert oal.oal_gated_prefill_workspace_bytes(2, 4, 2, 0) > 0
    assert oal.oal_gated_prefill_workspace_bytes(2, 4, 2, 4096) % 256 == 0
    assert oal.oal_gated_prefill_workspace_bytes(2, 4, 3, 4096) == 0
    assert oal.oal_gated_backward_workspace_bytes(2, 4, 2, 4096) % 256 == 0
    assert oal.oal_gated_backward_workspace_bytes(2, 4, 2, 4096, d=32) == 0


def test_binding_refuses_wrong_tensors(lib):
    from grouped_quadratic_gb300 import oal
    z = torch.zeros
    Q, K, g = z(1, 4, 8, 64), z(1, 2, 8, 64), z(1, 2, 8)
    cases = [
        lambda: oal.oal_gated_prefill(Q, K, K, g),                                   # CPU tensors
        lambda: oal.oal_gated_prefill(Q, K, K, g.double()),
        lambda: oal.oal_gated_prefill(Q, K.bfloat16(), K, g),
        lambda: oal.oal_gated_prefill(Q, K, K[:, :, :7], g),
        lambda: oal.oal_gated_prefill(Q[0], K, K, g),
        lambda: oal.oal_gated_prefill(Q, K, K, g, continue_from_state=True),         # from no state
        lambda: oal.oal_gated_backward(Q, K, K, g, Q[:, :2]),
        lambda: oal.oal_gated_decode_step(Q[:, :, 0], K[:, :, 0], K[:, :, 0], g[:, :, 0], z(1, 2, 64, 64)),
        lambda: oal.oal_gated_decode_step(Q, K, K, g, z(1, 2, 64, 64)),
        lambda: oal.oal_state_remap(z(4, 8), z(4, dtype=torch.int32)),
        lambda: oal.oal_state_remap(z(4, 8), z(3, dtype=torch.int32)),
    ]
    for call in cases:
        with pytest.raises(oal.OALError) as e:
            call()
        assert e.value.status == oal.OAL_ERR_INVALID_ARG


class FakeStream:
    """What the binding uses of a torch.cuda.Stream, with its calls in order."""
    device = torch.device("cuda", 0)
    cuda_stream = 4321

    def __init__(self):
        self.calls = []

    def wait_stream(self, other):
        self.calls.append(("wait", other))


class FakeTensor:
    def record_stream(self, stream):
        stream.calls.append(("record", self))


def test_tensors_made_in_a_call_are_ordered_before_its_stream(lib, monkeypatch):
    """A call makes (and fills) its tensors on the current stream; the stream it
    launches on has to wait for that, and the memory must live until it is done."""
    from grouped_quadratic_gb300 import oal
    now, side, made = FakeStream(), FakeStream(), [FakeTensor(), FakeTensor()]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now)
    assert oal._stream_on(now.device, side, made) == side.cuda_stream
    assert ("wait", now) in side.calls
    assert all(("record", t) in side.calls for t in made)
    # nothing made, or the current stream itself: no order to add
    side.calls.clear()
    assert oal._stream_on(now.device, side, []) == side.cuda_stream
    assert oal._stream_on(now.device, now, made) == now.cuda_stream
    assert side.calls == [] and now.calls == []
