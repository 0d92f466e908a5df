"""What beam selection, cache reordering and the 8-bit cache refuse before anything is enqueued.
No GPU is needed: every call here is turned down on the host (the pointers are never followed)."""
import ctypes

import pytest

from persistent_megakernel_interpreter_b200 import _lib

OK, INVALID, UNSUPPORTED = 0, 1, 3
PTR = ctypes.c_void_p(4096)


def select(**kw):
    a = dict(logits=PTR, ld=100, batch=1, beams=2, vocab=100, n_out=2, scores=PTR, finished=None, eos=-1, tokens=PTR,
             parents=PTR, out=PTR, next_finished=None, positions=None)
    a.update(kw)
    return _lib.lib().mk_beam_select(*a.values(), None)


@pytest.mark.parametrize("kw, code", [
    (dict(logits=None), INVALID), (dict(scores=None), INVALID), (dict(tokens=None), INVALID),
    (dict(parents=None), INVALID), (dict(out=None), INVALID), (dict(batch=0), INVALID), (dict(beams=0), INVALID),
    (dict(vocab=0), INVALID), (dict(n_out=0), INVALID), (dict(ld=99), INVALID), (dict(ld=-100), INVALID),
    (dict(vocab=1, ld=1, n_out=3), INVALID), (dict(beams=17), UNSUPPORTED), (dict(n_out=33), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1, ld=1 << 25), UNSUPPORTED), (dict(batch=(1 << 20) + 1), UNSUPPORTED),
    (dict(finished=PTR, eos=-1), INVALID), (dict(finished=PTR, eos=100), INVALID), (dict(next_finished=PTR), INVALID),
    (dict(logits=ctypes.c_void_p(4098)), INVALID)])
def test_beam_select_refuses(kw, code):
    assert select(**kw) == code


def config(**kw):
    a = dict(n_layers=2, hidden=0, n_heads=0, n_kv_heads=2, head_dim=64, ffn=0, vocab=0, rms_eps=0.0, rope_theta=0.0,
             max_batch=4, max_seq=64)
    a.update(kw)
    return ctypes.byref(_lib.MkConfig(*a.values()))


@pytest.mark.parametrize("cfg, k, v, rows, parents, lengths, code", [
    (None, PTR, PTR, 2, PTR, PTR, INVALID), ({}, None, PTR, 2, PTR, PTR, INVALID), ({}, PTR, None, 2, PTR, PTR, INVALID),
    ({}, PTR, PTR, 2, None, PTR, INVALID), ({}, PTR, PTR, 2, PTR, None, INVALID), ({}, PTR, PTR, 0, PTR, PTR, INVALID),
    ({}, PTR, PTR, 5, PTR, PTR, INVALID), ({}, ctypes.c_void_p(4104), PTR, 2, PTR, PTR, INVALID),
    ({"head_dim": 96}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED), ({"max_batch": 9}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED),
    ({"max_seq": 0}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED), ({"max_seq": (1 << 20) + 1}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED),
    ({"n_layers": 65}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED), ({"n_kv_heads": 0}, PTR, PTR, 2, PTR, PTR, UNSUPPORTED)])
def test_cache_reorder_refuses(cfg, k, v, rows, parents, lengths, code):
    c = None if cfg is None else config(**cfg)
    assert _lib.lib().mk_cache_reorder(c, k, v, rows, parents, lengths, None, None) == code


def qcache(**kw):
    a = dict(n_layers=2, max_batch=4, n_kv_heads=2, max_seq=2048, head_dim=64, reserved0=0, k_codes=4096, v_codes=4096,
             k_scale=4096, v_scale=4096, k_tail=4096, v_tail=4096)
    a.update(kw)
    return ctypes.byref(_lib.MkQcache(*a.values()))


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(v_tail=None), INVALID), (dict(k_scale=None), INVALID),
              (dict(k_codes=4104), INVALID), (dict(v_tail=4098), INVALID), (dict(v_scale=4098), INVALID),
              (dict(head_dim=32), UNSUPPORTED), (dict(max_batch=0), UNSUPPORTED), (dict(max_batch=9), UNSUPPORTED),
              (dict(n_kv_heads=33), UNSUPPORTED), (dict(n_layers=0), UNSUPPORTED), (dict(max_seq=0), UNSUPPORTED),
              (dict(max_seq=(1 << 20) + 1), UNSUPPORTED)]


def append(c, first=0, layers=1, rows=2, n_new=3, k=PTR, v=PTR, strides=(0, 384, 192, 64), positions=PTR):
    st = None if strides is None else (ctypes.c_int64 * 4)(*strides)
    return _lib.lib().mk_qcache_append(c, first, layers, rows, n_new, k, v, st, positions, None, None)


def attend(c, layer=0, rows=2, n_heads=4, max_ctx=64, q=PTR, positions=PTR, out=PTR, work=None, size=0):
    return _lib.lib().mk_qcache_attention(c, layer, rows, n_heads, max_ctx, q, positions, out, work, size, None)


@pytest.mark.parametrize("bad, code", BAD_CACHES)
def test_a_bad_cache_is_refused_by_every_call(bad, code):
    c = qcache(**bad)
    assert append(c) == code and attend(c) == code
    assert _lib.lib().mk_qcache_reorder(c, 2, PTR, PTR, None, None) == code
    assert _lib.lib().mk_qcache_attention_workspace(c, 2, 4, 2048) == 0
    assert _lib.lib().mk_qcache_reorder(None, 2, PTR, PTR, None, None) == INVALID


@pytest.mark.parametrize("kw", [dict(first=-1), dict(first=2), dict(first=1, layers=2), dict(layers=0), dict(rows=0),
                                dict(rows=5), dict(n_new=0), dict(n_new=2049), dict(k=None), dict(v=None),
                                dict(strides=None), dict(strides=(0, 384, 192, 4)), dict(positions=None),
                                dict(k=ctypes.c_void_p(4104)), dict(v=ctypes.c_void_p(4098))])
def test_append_refuses(kw):
    assert append(qcache(), **kw) == INVALID


@pytest.mark.parametrize("kw, code", [
    (dict(layer=-1), INVALID), (dict(layer=2), INVALID), (dict(rows=0), INVALID), (dict(rows=5), INVALID),
    (dict(max_ctx=0), INVALID), (dict(max_ctx=2049), INVALID), (dict(q=None), INVALID), (dict(positions=None), INVALID),
    (dict(out=None), INVALID), (dict(n_heads=3), UNSUPPORTED), (dict(n_heads=10), UNSUPPORTED), (dict(n_heads=0), UNSUPPORTED),
    (dict(max_ctx=2048), INVALID), (dict(max_ctx=2048, work=PTR, size=1024), INVALID),
    (dict(max_ctx=2048, work=ctypes.c_void_p(4104), size=1 << 30), INVALID)])
def test_attention_refuses(kw, code):
    assert attend(qcache(), **kw) == code


def test_workspace_is_asked_for_only_where_it_is_used():
    ask = _lib.lib().mk_qcache_attention_workspace
    assert ask(qcache(), 2, 4, 32) == 0
    assert ask(qcache(), 2, 4, 2048) > 0
    assert ask(qcache(), 2, 3, 2048) == 0 and ask(qcache(), 5, 4, 2048) == 0 and ask(qcache(), 2, 4, 4096) == 0


@pytest.mark.parametrize("rows, parents, lengths", [(0, PTR, PTR), (5, PTR, PTR), (2, None, PTR), (2, PTR, None)])
def test_qcache_reorder_refuses(rows, parents, lengths):
    assert _lib.lib().mk_qcache_reorder(qcache(), rows, parents, lengths, None, None) == INVALID


def test_step_on_the_8_bit_cache_refuses_without_a_handle():
    assert _lib.lib().mk_decode_step_qcache(None, qcache(), 1, 64, PTR, PTR, PTR, PTR, 1 << 30, None, None) == INVALID
    assert _lib.lib().mk_decode_step_qcache_workspace(None, qcache(), 1, 64) == 0


def test_cache_struct_matches_the_c_header(tmp_path):
    import os
    import shutil
    import subprocess
    from conftest import ROOT
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    fields = [n for n, _ in _lib.MkQcache._fields_]
    src = tmp_path / "q.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mk.h"\nint main(void) {\n'
                   '    printf("%zu %d", sizeof(mk_qcache), MK_QCACHE_BLOCK);\n'
                   + "".join(f'    printf(" %zu", offsetof(mk_qcache, {f}));\n' for f in fields) + "    return 0;\n}\n")
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Werror", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o",
                           str(tmp_path / "q")])
    got = [int(x) for x in subprocess.run([str(tmp_path / "q")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(_lib.MkQcache), _lib.QCACHE_BLOCK] + [getattr(_lib.MkQcache, f).offset for f in fields]


def test_compiled_binding_refuses_before_it_calls():
    """Host tensors, wrong kinds of arguments and wrong counts of them raise; no CUDA device is asked for."""
    import torch
    call = _lib.call()
    x, s, t = torch.zeros(2, 8), torch.zeros(1, 2), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(AssertionError, match="logits"):
        call.beam_select(x, s, t, t, s, None, -1, None, None, None)
    with pytest.raises(AssertionError, match="logits: a tensor"):
        call.beam_select(None, s, t, t, s, None, -1, None, None, None)
    with pytest.raises(TypeError):
        call.beam_select(x, s)
    with pytest.raises(AssertionError, match="k_cache"):
        call.cache_reorder(x, x, t, t, None, None)
    c = _lib.MkQcache(1, 1, 1, 64, 64, 0, *([4096] * 6))
    at = ctypes.addressof(c)
    with pytest.raises(AssertionError, match="k: "):
        call.qcache_append(at, 0, x, x, t, None, 0, None)
    with pytest.raises(AssertionError, match="parents"):
        call.qcache_reorder(at, 0, t, t, None, None)
    with pytest.raises(AssertionError, match="q: "):
        call.qcache_attention(at, 0, 0, x, t, x, 64, None, None)


def test_missing_binding_fails_loudly(monkeypatch, tmp_path):
    monkeypatch.setattr(_lib, "_call", None)
    monkeypatch.setattr(_lib, "_HERE", str(tmp_path))
    with pytest.raises(RuntimeError, match="missing"):
        _lib.call()
