"""Which stream a call of the binding runs on: the current one of its tensors' device, whichever of its buffers is a tensor and
whichever an address.  The library's functions are stood in for; nothing is launched."""

import pytest

import torch

import tiled_movement_amd as T
from test_feed_forward_host import A, B, BF, BYTE, C, CALLS, D, E, FL, WS, Placed

STREAM = 0x51AB0


@pytest.fixture
def seen(monkeypatch):
    """The stream arguments of the calls that reach the library."""
    got = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(T, "_raw_stream", lambda index: STREAM + index)
    for name in T.EXPORTS:
        if hasattr(T, name) and not name.endswith("workspace"):
            monkeypatch.setattr(T.lib, name, lambda *a: got.append(a[-1]) or T.SWZ_OK)
    return got


@pytest.mark.parametrize("name", CALLS)
def test_any_buffer_names_the_stream(seen, name):
    types, call, _ = CALLS[name]
    address = {buf: A + (i << 36) for i, buf in enumerate(types)}
    call(dict(address), {})
    assert seen == [None]  # addresses alone: the NULL stream
    for buf in types:
        call({**address, buf: Placed(address[buf], types[buf], 1 << 24)}, {})
        assert seen[-1] == STREAM, buf
        call({**address, buf: Placed(address[buf], types[buf], 1 << 24)}, {"stream": 0x77})
        assert seen[-1] == 0x77


@pytest.mark.parametrize("as_list", [list, iter, tuple])
def test_norm_calls_run_on_their_tensors_stream(seen, as_list):
    """norm and ws as addresses: the tensors of the list are what the stream has to wait for."""
    tensors = [Placed(A, BF, 200), Placed(B, FL, 400)]
    to = [Placed(E, BF, 200), Placed(C, FL, 400)]
    for norm in (D, Placed(D, FL, 8)):
        for ws in (WS, Placed(WS, BYTE, 1 << 20)):
            T.swz_grad_norm(as_list(tensors), norm, ws)
            T.swz_clip_grads(as_list(tensors), 1.0, norm, ws)
            T.swz_clip_grads(as_list(tensors), 1.0, norm, ws, out=as_list(to))
            assert seen[-3:] == [STREAM] * 3
    T.swz_grad_norm(as_list(tensors), D, WS, stream=0x77)
    T.swz_clip_grads([], 1.0, Placed(D, FL, 8), None)
    assert seen[-2:] == [0x77, STREAM]
