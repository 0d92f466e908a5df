"""Contracts of beam selection, reordering and the 8-bit cache that hold on the host, before anything is enqueued: calls
that are refused (no pointer is followed), and what the binding checks. No GPU is needed."""
import ctypes

import pytest

from persistent_megakernel_interpreter_b200 import _lib

OK, INVALID, UNSUPPORTED = 0, 1, 3
PTR = ctypes.c_void_p(4096)


def qcache(**kw):
    a = dict(n_layers=2, max_batch=4, n_kv_heads=2, max_seq=2048, head_dim=64, reserved0=0, k_codes=4096, v_codes=4096,
             k_scale=4096, v_scale=4096, k_tail=4096, v_tail=4096)
    a.update(kw)
    return ctypes.byref(_lib.MkQcache(*a.values()))


@pytest.mark.parametrize("kw, code", [
    (dict(lengths=None), INVALID), (dict(positions=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(layer=2), INVALID), (dict(rows=5), INVALID), (dict(max_ctx=2049), INVALID), (dict(n_heads=10), UNSUPPORTED),
    (dict(max_ctx=2048), INVALID), (dict(cache=dict(head_dim=32)), UNSUPPORTED)])
def test_attention_of_a_prefix_refuses(kw, code):
    a = dict(cache={}, layer=0, rows=2, n_heads=4, max_ctx=64, q=PTR, positions=PTR, lengths=PTR, out=PTR, work=None, size=0)
    a.update(kw)
    a["cache"] = qcache(**a["cache"])
    assert _lib.lib().mk_qcache_attention_prefix(*a.values(), None) == code


def test_a_checked_selection_refuses_without_a_status():
    def call(logits, status):
        return _lib.lib().mk_beam_select_checked(logits, 100, 1, 2, 100, 2, PTR, None, -1, PTR, PTR, PTR, None, None, status, None)
    assert call(PTR, None) == INVALID and call(None, PTR) == INVALID
    assert _lib.lib().mk_device_status(None) is None


def test_a_cache_on_another_device_than_the_model_is_refused(monkeypatch):
    """Before the library is called or anything is allocated: its pointers would be followed on the wrong device."""
    from types import SimpleNamespace
    import torch
    from persistent_megakernel_interpreter_b200.config import TINY
    from persistent_megakernel_interpreter_b200.model import Megakernel
    mk = Megakernel.__new__(Megakernel)
    mk._h, mk.device, mk.cfg, mk.max_seq = None, 0, TINY, 64
    cache = SimpleNamespace(_device=1, _ref=None, max_seq=64)

    def called(*a):
        raise RuntimeError("reached")
    monkeypatch.setattr(_lib, "lib", lambda: SimpleNamespace(mk_decode_step_qcache=called, mk_decode_step_qcache_workspace=called))
    x = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(AssertionError, match="cuda:1"):
        mk.decode_step_qcache_workspace(cache, 1, 64)
    for ws in (None, x):
        with pytest.raises(AssertionError, match="cuda:1"):
            mk.decode_step_qcache(x, x, cache, x, workspace=ws)
    cache._device = 0
    with pytest.raises(RuntimeError, match="reached"):
        mk.decode_step_qcache_workspace(cache, 1, 64)


@pytest.mark.parametrize("batch, beams, n_out, scores, finished, code", [
    (2, 4, 2, True, False, INVALID), (2, 4, 8, True, False, INVALID), (2, 4, 2, False, True, INVALID), (3, 2, 1, True, True, INVALID)])
def test_a_selection_in_place_refuses_where_sequences_would_overlap(batch, beams, n_out, scores, finished, code):
    """Sequence b's results at b * n_out would lie among the scores of another, which may still be read."""
    other = ctypes.c_void_p(1 << 20)
    got = _lib.lib().mk_beam_select(PTR, 100, batch, beams, 100, n_out, PTR, PTR, 5, other, other, PTR if scores else other,
                                    PTR if finished else other, None, None)
    assert got == code


@pytest.mark.parametrize("apart, code", [(0, INVALID), (16, INVALID), (-16, INVALID), (131056, INVALID), (-131056, INVALID)])
def test_reorder_refuses_caches_that_overlap(apart, code):
    """Keys and values are moved by the same launch: where they overlap, a slot would be read and written by two threads.
    One cache here is 2 x 4 x 2 x 64 x 64 elements, 131072 bytes."""
    cfg = _lib.MkConfig(2, 0, 0, 2, 64, 0, 0, 0.0, 0.0, 4, 64)
    at = 1 << 20
    assert _lib.lib().mk_cache_reorder(ctypes.byref(cfg), at, at + apart, 2, PTR, PTR, None, None) == code


def test_a_status_that_is_no_tensor_is_refused():
    """A number would be taken for a device address."""
    import torch
    from persistent_megakernel_interpreter_b200.model import beam_select
    x, s, t = torch.zeros(2, 8), torch.zeros(1, 2), torch.zeros(1, 2, dtype=torch.int32)
    for bad in (1, 0, 4096, True):
        with pytest.raises(AssertionError, match="status"):
            beam_select(x, s, t, t, s, status=bad)
