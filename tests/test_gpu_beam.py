"""Beam selection and cache reordering on the GPU against plain 64-bit forms, and beam search over decode steps.

Tokens, parents and copied slots are exact. A score is off by the rounding of the fp32 sum and of the result: the sum's
relative error is at most (vocab / 512 + 64) 2^-24 (that many additions behind one another at most) plus
17 * 2^-23 for the exponents' arguments and 2^-21 for the exponential itself, which is the logarithm's absolute error;
rounding the result adds 2^-24 of its magnitude."""
import numpy as np
import pytest
import torch

from cases_beam_cache import reorder, select
from persistent_megakernel_interpreter_b200.config import TINY
from persistent_megakernel_interpreter_b200.inputs import make_kv_cache, make_tokens, make_weights
from persistent_megakernel_interpreter_b200.model import Megakernel, beam_select, cache_reorder

pytestmark = pytest.mark.gpu


def score_tol(vocab, total):
    return (vocab / 512 + 64) * 2.0 ** -24 + 17 * 2.0 ** -23 + 2.0 ** -21 + np.abs(total) * 2.0 ** -24


def gpu_select(x, scores, n_out, finished=None, eos=-1, offset=0, stride=None, positions=None, in_place=False):
    rows, vocab = x.shape
    stride = stride or vocab
    buf = torch.full((offset + rows * stride + 8,), 50.0, device="cuda")
    logits = buf[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    logits.copy_(torch.from_numpy(x))
    sc = torch.from_numpy(scores).cuda()
    fin = None if finished is None else torch.from_numpy(finished.astype(np.int32)).cuda()
    batch = scores.shape[0]
    tok = torch.full((batch, n_out), -7, dtype=torch.int32, device="cuda")
    par = torch.full((batch, n_out), -7, dtype=torch.int32, device="cuda")
    out = sc if in_place else torch.full((batch, n_out), 7.0, device="cuda")
    nf = None if fin is None else fin if in_place else torch.full((batch, n_out), -7, dtype=torch.int32, device="cuda")
    beam_select(logits, sc, tok, par, out, finished=fin, eos=eos, next_finished=nf, positions=positions)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (tok, par, out, nf)]


def check(x, scores, n_out, finished=None, eos=-1, **kw):
    tok, par, tot, fin = select(x, scores, n_out, finished, eos)
    got = gpu_select(x, scores, n_out, finished, eos, **kw)
    assert np.array_equal(got[0], tok) and np.array_equal(got[1], par)
    ends = np.isfinite(tot)
    assert np.array_equal(got[2][~ends], tot[~ends].astype(np.float32))
    assert np.all(np.abs(got[2][ends] - tot[ends]) <= score_tol(x.shape[1], tot[ends]))
    if finished is not None:
        assert np.array_equal(got[3], fin)


def draw(batch, beams, vocab, seed):
    g = np.random.default_rng(seed)
    return g.standard_normal((batch * beams, vocab)).astype(np.float32) * 3, \
        -g.random((batch, beams)).astype(np.float32) * 9, g


@pytest.mark.parametrize("vocab", [1, 3, 33, 1001, 4096, 50257, 128256])
@pytest.mark.parametrize("batch, beams, n_out", [(1, 1, 1), (1, 4, 8), (2, 3, 3), (3, 5, 10), (1, 16, 32), (40, 2, 4)])
def test_beam_select_against_the_plain_form(batch, beams, n_out, vocab):
    if batch * beams * vocab > 6_000_000:
        pytest.skip("the 64-bit form of this size takes long")
    x, scores, _ = draw(batch, beams, vocab, vocab + beams)
    check(x, scores, min(n_out, beams * vocab))


@pytest.mark.parametrize("batch, beams, vocab, n_out", [(33, 3, 20011, 6), (5, 1, 128256, 8), (2, 9, 30001, 18), (1, 7, 128256, 14),
                                                         (3, 13, 1000, 32), (129, 16, 300, 4), (64, 1, 9001, 1)])
def test_every_way_of_cutting_the_rows(batch, beams, vocab, n_out):
    x, scores, g = draw(batch, beams, vocab, batch)
    check(x, scores, n_out)
    fin = (g.random((batch, beams)) < 0.4).astype(np.int32)
    check(x, scores, n_out, fin, eos=vocab - 1)


@pytest.mark.parametrize("offset, stride", [(0, 1004), (1, 1001), (2, 1003), (3, 1024)])
def test_rows_of_any_alignment_and_stride(offset, stride):
    x, scores, _ = draw(2, 4, 1001, 5)
    check(x, scores, 8, offset=offset, stride=stride)


@pytest.mark.parametrize("vocab", [7, 4096, 50257])
def test_equal_rows_tie_to_the_lower_beam_and_equal_logits_to_the_lower_token(vocab):
    x, scores, g = draw(1, 4, vocab, 3)
    x[2] = x[0]
    x[3] = x[0]
    scores[0] = scores[0, 0]
    x[:, g.choice(vocab, 5, replace=False)] = 9.0
    check(x, scores, 12, offset=1)
    check(np.zeros_like(x), scores, 16)                  # nothing but ties
    check(np.round(x), scores, 16)                       # many of them


@pytest.mark.parametrize("vocab", [40, 5000, 128256])
def test_masks_infinities_and_nans(vocab):
    x, scores, g = draw(2, 4, vocab, 11)
    x[0] = -np.inf                                       # nothing left
    x[1, g.choice(vocab, vocab - 3, replace=False)] = -np.inf
    x[2] = np.finfo(np.float32).min                      # masked by the type's lowest value
    x[2, vocab // 2] = 1.0
    x[3, g.choice(vocab, vocab // 2, replace=False)] = np.nan
    x[4, [2, vocab - 1]] = np.inf
    x[5] = np.nan
    x[6] = np.finfo(np.float32).min
    x[7, :vocab // 3] = -np.inf
    scores[1, 3] = -np.inf                               # a beam not in use
    check(x, scores, 8)
    check(x, np.full_like(scores, -np.inf), 8)           # none in use: the lowest beams' best, at -infinity
    first = np.full_like(scores, -np.inf)
    first[:, 0] = 0.0                                    # the first step of a search
    check(x, first, 8)


def test_scores_that_are_no_numbers():
    x, scores, _ = draw(1, 4, 1000, 13)
    scores[0] = [np.nan, -np.inf, np.inf, -2.0]
    check(x, scores, 6)
    scores[0] = [np.nan, np.nan, -np.inf, np.finfo(np.float32).min]
    check(x, scores, 6)
    scores[0] = -1e30                                    # so far down that totals of one beam are equal
    check(x, scores, 6)


def test_the_best_logits_all_in_one_place():
    """Everything above the bound sits with a few threads: more is gathered than the list holds."""
    vocab = 128256
    x, scores, g = draw(1, 1, vocab, 23)
    at = (np.arange(vocab) // 4) % 512
    hot = at < 64                                        # the first two warps' tokens, 16032 of them
    x[0, hot] += 100.0
    check(x, scores, 32)
    x[0, hot] = 77.0                                     # and all of them equal
    check(x, scores, 32)
    x[0, hot] = 77.0 + (np.arange(vocab)[hot] % 7).astype(np.float32)
    check(x, scores, 32)


def test_finished_beams():
    x, scores, _ = draw(3, 4, 1001, 31)
    fin = np.array([[0, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 0]])
    scores[0, 1] = -0.25
    x[2, 500] = 60.0                                     # an unfinished beam that chooses eos
    x[4:8] = np.nan                                      # a finished sequence's rows are not looked at
    for n in (1, 4, 8, 32):
        check(x, scores, n, fin, eos=500)
    check(x, scores, 4, fin, eos=0)
    check(x, scores, 8, fin, eos=1000)
    check(x[:, :5].copy(), scores, 20, fin, eos=2)


def test_in_place_scores_and_positions():
    x, scores, _ = draw(2, 4, 4096, 41)
    fin = np.array([[0, 1, 0, 0], [0, 0, 0, 0]])
    pos = torch.arange(8, dtype=torch.int32, device="cuda") * 3
    check(x, scores, 4, fin, eos=9, in_place=True, positions=pos)
    assert np.array_equal(pos.cpu().numpy(), np.arange(8) * 3 + 1)


def test_select_captured_and_replayed():
    x, scores, _ = draw(2, 4, 4096, 43)
    y, _, _ = draw(2, 4, 4096, 44)
    logits, sc = torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda()
    tok = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    par, out = torch.zeros_like(tok), torch.zeros(2, 4, device="cuda")
    beam_select(logits, sc, tok, par, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beam_select(logits, sc, tok, par, out)
    logits.copy_(torch.from_numpy(y))
    graph.replay()
    torch.cuda.synchronize()
    t, p, _, _ = select(y, scores, 4)
    assert np.array_equal(tok.cpu().numpy(), t) and np.array_equal(par.cpu().numpy(), p)


def test_logits_written_by_the_kernel_just_before():
    """The selection is placed while the kernel before it ends; what that one wrote has to be seen."""
    for batch, vocab in ((2, 50257), (40, 4096)):
        sets = [torch.randn(batch * 4, vocab, device="cuda") for _ in range(3)]
        scores = torch.zeros(batch, 4, device="cuda")
        logits = torch.empty_like(sets[0])

        def outs():
            return [torch.zeros(batch, 8, dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.zeros(batch, 8, device="cuda")]

        want = []
        for x in sets:
            o = outs()
            beam_select(x, scores, *o)
            torch.cuda.synchronize()
            want.append(o)
        got = [outs() for _ in range(150)]
        for i, o in enumerate(got):
            logits.fill_(1.0)
            logits.copy_(sets[i % 3])
            beam_select(logits, scores, *o)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for i, o in enumerate(got) for a, b in zip(o, want[i % 3]))


# ------------------------------------------------------------------ reordering

def test_reorder_captured_and_replayed_with_other_parents():
    g = np.random.default_rng(2)
    shape = (2, 4, 2, 100, 64)
    k0, v0 = (torch.from_numpy(g.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16)).cuda() for _ in range(2))
    k, v = k0.clone(), v0.clone()
    par, n = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    par.copy_(torch.tensor([-1, 9, 2, 3]))                   # nobody moves
    cache_reorder(k.view(torch.bfloat16), v.view(torch.bfloat16), par, n)
    torch.cuda.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache_reorder(k.view(torch.bfloat16), v.view(torch.bfloat16), par, n)
    for parents, lengths in (([1, 0, 0, 3], [50, 100, 7, 9]), ([3, 3, 3, 3], [100, 1, 1, 64])):
        k.copy_(k0)
        v.copy_(v0)
        par.copy_(torch.tensor(parents))
        n.copy_(torch.tensor(lengths))
        graph.replay()
        torch.cuda.synchronize()
        for got, old in ((k, k0), (v, v0)):
            assert np.array_equal(got.cpu().numpy(), reorder(old.cpu().numpy(), parents, lambda p, r: (0, lengths[p])))


@pytest.mark.parametrize("layers, rows_of, heads, max_seq, dim", [(2, 4, 2, 160, 64), (1, 8, 8, 77, 128), (3, 1, 1, 5, 64),
                                                               (2, 5, 3, 1030, 64), (28, 8, 2, 33, 128)])
def test_cache_reorder_against_the_plain_form(layers, rows_of, heads, max_seq, dim):
    g = np.random.default_rng(max_seq)
    shape = (layers, rows_of, heads, max_seq, dim)
    k0, v0 = (g.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16) for _ in range(2))
    for trial in range(6):
        rows = rows_of if trial % 2 else max(1, rows_of - 1)
        parents = g.integers(0, rows, rows) if trial < 4 else g.permutation(rows)
        lengths = g.integers(0, max_seq + 1, rows)
        starts = None if trial == 0 else g.integers(0, max_seq + 1, rows)
        if trial == 3:
            parents[0], lengths[-1] = -1, max_seq + 50       # left alone; clamped
            starts[-1] = -4
        k, v = (torch.from_numpy(t).cuda().view(torch.bfloat16) for t in (k0, v0))
        i32 = [None if t is None else torch.as_tensor(t, dtype=torch.int32).cuda() for t in (parents, lengths, starts)]
        cache_reorder(k, v, i32[0], i32[1], starts=i32[2])
        torch.cuda.synchronize()
        n = np.clip(lengths, 0, max_seq)
        s = np.zeros(rows, int) if starts is None else np.clip(starts, 0, max_seq)
        for got, old in ((k, k0), (v, v0)):
            assert np.array_equal(got.view(torch.int16).cpu().numpy(), reorder(old, parents, lambda p, r: (s[r], n[p])))


def test_cache_reorder_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes: rows swapped behind the 4 GB mark are found where they belong."""
    shape = (2, 2, 4, 1 << 17, 128)
    k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    k[1, 0, 3, -3:] = 3.0
    k[1, 1, 3, -3:] = 5.0
    v = torch.zeros_like(k)
    v[1, 1, 0, 7] = 2.0
    parents = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    lengths = torch.full((2,), 1 << 17, dtype=torch.int32, device="cuda")
    cache_reorder(k, v, parents, lengths)
    assert torch.all(k[1, 0, 3, -3:] == 5) and torch.all(k[1, 1, 3, -3:] == 3)
    assert torch.all(v[1, 0, 0, 7] == 2) and torch.all(v[1, 1, 0, 7] == 0)
    assert int((k != 0).sum()) == 6 * 128 and int((v != 0).sum()) == 128


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("sequences, beams, use_eos", [(1, 4, False), (2, 3, True)])
def test_beam_search_over_decode_steps(sequences, beams, use_eos):
    """decode_steps_beam against the same steps with the choice and the copies made on the host: the logits are the
    same bits, so the tokens, parents, caches and scores have to agree."""
    rows, steps, past, max_seq = sequences * beams, 12, 20, 64
    w = make_weights(TINY, seed=3)
    k, v = make_kv_cache(TINY, rows, max_seq, past=past, seed=4)
    for t in (k, v):                                        # the beams of a sequence share its prompt
        for r in range(rows):
            t[:, r] = t[:, r // beams * beams]
    mk = Megakernel(TINY, w.to("cuda"), max_batch=rows, max_seq=max_seq)
    mk.build_schedule(rows, max_seq)
    tok0 = make_tokens(TINY, sequences, seed=5).repeat_interleave(beams).to(torch.int32).cuda()
    sc0 = torch.full((sequences, beams), -float("inf"))
    sc0[:, 0] = 0.0
    start = torch.full((rows,), past, dtype=torch.int32, device="cuda")

    def state():
        return (tok0.clone(), start.clone(), k.cuda(), v.cuda(), torch.empty(rows, TINY.vocab, device="cuda"), sc0.cuda(),
                torch.zeros(sequences, beams, dtype=torch.int32, device="cuda"))

    eos = -1
    hist = None
    for attempt in range(2 if use_eos else 1):
        tok, pos, kd, vd, lg, sc, fin = state()
        gen = torch.zeros(steps, rows, dtype=torch.int32, device="cuda")
        par = torch.zeros(steps, rows, dtype=torch.int32, device="cuda")
        mk.decode_steps_beam(tok, pos, (kd, vd), lg, sc, steps, finished=fin if eos >= 0 else None, eos=eos, starts=start,
                             generated=gen, parents=par)
        torch.cuda.synchronize()
        assert mk.status()[0] == 0
        hist = gen.cpu().numpy()
        if use_eos and attempt == 0:
            eos = int(hist[2, 0])                           # a token that is chosen on the way
    t2, p2, k2, v2, l2, s2, f2 = state()
    s2, f2 = s2.cpu().numpy(), f2.cpu().numpy()
    par = par.cpu().numpy()
    for i in range(steps):
        mk.decode_step(t2, p2, k2, v2, l2)
        torch.cuda.synchronize()
        t, p, s, f = select(l2.cpu().numpy(), s2, beams, f2 if eos >= 0 else None, eos)
        assert np.array_equal(hist[i], t.reshape(-1)) and np.array_equal(par[i], p.reshape(-1)), i
        s2, f2 = s.astype(np.float32), f
        t2 = torch.as_tensor(t.reshape(-1), dtype=torch.int32).cuda()
        p2 = p2 + 1
        at = torch.as_tensor(p.reshape(-1)).cuda()
        k2, v2 = k2[:, at].contiguous(), v2[:, at].contiguous()
    n = past + steps
    assert torch.equal(kd[:, :, :, :n], k2[:, :, :, :n]) and torch.equal(vd[:, :, :, :n], v2[:, :, :, :n])
    assert torch.equal(pos, p2)
    assert np.all(np.abs(sc.cpu().numpy() - s2) <= steps * score_tol(TINY.vocab, s2))
    if eos >= 0:
        assert np.array_equal(fin.cpu().numpy(), f2) and f2.any()
    mk.close()
