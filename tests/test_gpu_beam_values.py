"""Beam selection where the logits are not the ordinary ones, against the plain 64-bit form: tokens and parents are exact; a
score is off by at most the fp32 sum's rounding, (vocab / 512 + 64) 2^-24 + 17 * 2^-23 + 2^-21 in its logarithm, and 2^-24 of
its magnitude."""
import numpy as np
import pytest
import torch

from cases_beam_cache import select
from persistent_megakernel_interpreter_b200.model import beam_select

pytestmark = pytest.mark.gpu

BIG = np.finfo(np.float32).max


def check(x, scores, n_out):
    tok, par, tot, _ = select(x, scores, n_out)
    got = [torch.full((scores.shape[0], n_out), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    got.append(torch.full((scores.shape[0], n_out), 7.0, device="cuda"))
    beam_select(torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda(), *got)
    torch.cuda.synchronize()
    t, p, s = (g.cpu().numpy() for g in got)
    assert np.array_equal(t, tok) and np.array_equal(p, par)
    ends = np.isfinite(tot)
    assert np.array_equal(s[~ends], tot[~ends].astype(np.float32))
    tol = (x.shape[1] / 512 + 64) * 2.0 ** -24 + 17 * 2.0 ** -23 + 2.0 ** -21 + np.abs(tot[ends]) * 2.0 ** -24
    assert np.all(np.abs(s[ends] - tot[ends]) <= tol)


@pytest.mark.parametrize("batch, beams, vocab", [(1, 1, 128256), (2, 4, 128256), (1, 4, 4096), (40, 4, 1000), (3, 16, 300)])
def test_infinite_logits_beside_the_largest_number(batch, beams, vocab):
    """The infinite ones share their row among themselves, wherever the row is cut."""
    g = np.random.default_rng(vocab)
    x = g.standard_normal((batch * beams, vocab)).astype(np.float32)
    scores = np.zeros((batch, beams), np.float32)
    for r in range(batch * beams):
        x[r, g.choice(vocab, 40, replace=False)] = BIG
        x[r, g.choice(vocab, 1 + r % 3, replace=False)] = np.inf
    check(x, scores, min(8, vocab))
    x[:, vocab // 2:] = BIG                                  # half of each row
    x[:, 1] = np.inf
    check(x, scores, min(8, vocab))
    x[:, 1] = -np.inf                                        # and without infinities
    x[np.isposinf(x)] = BIG
    check(x, scores, min(8, vocab))


@pytest.mark.parametrize("batch, beams, n_out", [(1, 6, 2), (1, 6, 6), (5, 3, 3)])
def test_in_place_where_it_is_allowed(batch, beams, n_out):
    g = np.random.default_rng(beams)
    x, scores = g.standard_normal((batch * beams, 2000)).astype(np.float32), -g.random((batch, beams)).astype(np.float32)
    fin = g.random((batch, beams)) < 0.3
    tok, par, tot, nf = select(x, scores, n_out, fin, 9)
    sc, f = torch.from_numpy(scores).cuda(), torch.from_numpy(fin.astype(np.int32)).cuda()
    t, p = (torch.zeros(batch, n_out, dtype=torch.int32, device="cuda") for _ in range(2))
    beam_select(torch.from_numpy(x).cuda(), sc, t, p, sc, finished=f, eos=9, next_finished=f)
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), tok) and np.array_equal(p.cpu().numpy(), par)
    assert np.array_equal(f.view(-1)[:batch * n_out].cpu().numpy().reshape(batch, n_out), nf)
    assert np.allclose(sc.view(-1)[:batch * n_out].cpu().numpy().reshape(batch, n_out), tot, rtol=2e-6, atol=1e-5)


# pieces of a row and threads that take a piece's tokens in turn, by the launch's rule
CUTS = [(1, 1, 128256, 8, 256), (2, 4, 128256, 4, 512), (1, 1, 49000, 8, 128), (5, 8, 20000, 1, 512)]


@pytest.mark.parametrize("batch, beams, vocab, pieces, threads", CUTS)
@pytest.mark.parametrize("n_out, share", [(32, 30 / 128), (8, 7 / 32)])
def test_more_above_the_bound_than_the_list_holds(batch, beams, vocab, pieces, threads, n_out, share):
    """Everything that is large sits with a few of a piece's threads, fewer than n_out of the groups whose maxima give the bound:
    the bound is one of the small numbers, thousands lie above it, and it has to be raised."""
    g = np.random.default_rng(vocab + n_out)
    size = -(-vocab // pieces)
    hot = np.arange(vocab) % size % threads < int(share * threads)
    x = g.standard_normal((batch * beams, vocab)).astype(np.float32)
    scores = -g.random((batch, beams)).astype(np.float32)
    x[:, hot] += 100.0
    check(x, scores, n_out)                                  # all of them different
    x[:, hot] = np.sort(x[:, hot], axis=1)
    check(x, scores, n_out)                                  # in order: the largest at the end
    x[:, hot] = 77.0 + (np.arange(hot.sum()) % 2).astype(np.float32)
    check(x, scores, n_out)                                  # half of them the largest
    x[:, hot] = 77.0 + (np.arange(hot.sum()) % 500 == 3).astype(np.float32)
    check(x, scores, n_out)                                  # a few the largest, the others equal
    x[:, hot] = 77.0 + np.minimum(np.arange(hot.sum()), 40).astype(np.float32)
    check(x, scores, n_out)
