"""Beam search over decode steps that fail, or whose buffers are larger than the step, on both kinds of cache. Tokens, parents,
positions, scores and caches are compared for equality with a search that stops in time."""
import numpy as np
import pytest
import torch

from persistent_megakernel_interpreter_b200.config import TINY
from persistent_megakernel_interpreter_b200.inputs import make_kv_cache, make_tokens, make_weights
from persistent_megakernel_interpreter_b200.model import Megakernel, beam_select
from persistent_megakernel_interpreter_b200.qcache import QCache

pytestmark = pytest.mark.gpu

BAD_TOKEN, BAD_POSITION = 6, 7


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Search:
    """Two sequences of two beams; the second is further on than the first."""

    def __init__(self, kind, max_seq=64, past=(10, 60), max_batch=4):
        self.kind, rows = kind, 4
        self.mk = Megakernel(TINY, make_weights(TINY, seed=3).to("cuda"), max_batch=max_batch, max_seq=max_seq)
        lengths = [past[0]] * 2 + [past[1]] * 2
        k, v = make_kv_cache(TINY, max_batch, max_seq, past=lengths + [0] * (max_batch - rows), seed=4)
        if kind == "8-bit":
            self.cache = QCache(TINY, max_batch, max_seq)
            self.cache.append(k.cuda()[:, :rows], v.cuda()[:, :rows], i32([0] * rows), counts=i32(lengths))
            self.held = [self.cache.k_codes, self.cache.v_codes, self.cache.k_scale, self.cache.v_scale, self.cache.k_tail,
                         self.cache.v_tail]
        else:
            self.mk.build_schedule(rows, max_seq)
            self.held = [k.cuda(), v.cuda()]
            self.cache = tuple(self.held)
        self.tokens, self.positions = make_tokens(TINY, rows, seed=5).to(torch.int32).cuda(), i32(lengths)
        self.starts = self.positions.clone()
        self.scores = torch.zeros(2, 2, device="cuda")
        self.logits = torch.empty(rows, TINY.vocab, device="cuda")
        self.finished = torch.zeros(2, 2, dtype=torch.int32, device="cuda")

    def run(self, steps, **kw):
        gen, par = (torch.full((steps, 4), 9, dtype=torch.int32, device="cuda") for _ in range(2))
        self.mk.decode_steps_beam(self.tokens, self.positions, self.cache, self.logits, self.scores, steps, finished=self.finished,
                                  eos=7, starts=self.starts, generated=gen, parents=par, **kw)
        torch.cuda.synchronize()
        return gen, par

    def state(self):
        return [t.clone() for t in (self.tokens, self.positions, self.scores, self.finished, *self.held)]

    def code(self, status):
        return int(status.item()) if self.kind == "8-bit" else self.mk.status()[0]


@pytest.mark.parametrize("kind", ["8-bit", "bf16"])
def test_a_row_at_the_end_of_the_cache_ends_the_search_there(kind):
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    kw = {"status": status} if kind == "8-bit" else {}
    a, b = Search(kind), Search(kind)
    gen_a, par_a = a.run(4, **kw)                            # positions 60 .. 63: as many as fit
    assert a.code(status) == 0
    gen_b, par_b = b.run(9, **kw)                            # the fifth finds no slot
    assert b.code(status) == BAD_POSITION
    assert torch.equal(gen_a, gen_b[:4]) and torch.equal(par_a, par_b[:4])
    assert torch.all(par_b[4:] == -1) and torch.equal(gen_b[4:], a.tokens.expand(5, 4))
    assert b.positions.tolist() == [14, 14, 64, 64]
    assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    # the other sequence goes on once the rows that are at the end stand elsewhere (the start of a block)
    before = b.state()
    b.positions[2:] = 32
    b.starts[2:] = 32
    gen, par = b.run(2, **kw)
    assert b.code(status) == 0 and torch.all(par >= 0) and b.positions.tolist() == [16, 16, 34, 34]
    assert not torch.equal(b.state()[2], before[2])
    a.mk.close()
    b.mk.close()


@pytest.mark.parametrize("kind", ["8-bit", "bf16"])
def test_a_bad_token_changes_nothing(kind):
    for with_status in ((True, False) if kind == "8-bit" else (False,)):
        s = Search(kind)
        s.tokens[1] = TINY.vocab
        s.logits.copy_(torch.randn(4, TINY.vocab))           # of an earlier step, it might seem
        before = s.state()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gen, par = s.run(3, **({"status": status} if with_status else {}))
        assert torch.all(par == -1)
        assert all(torch.equal(x, y) for x, y in zip(before, s.state()))
        if with_status or kind == "bf16":
            assert s.code(status) == BAD_TOKEN
        s.mk.close()


def test_status_belongs_to_the_8_bit_cache():
    s = Search("bf16")
    with pytest.raises(AssertionError, match="status"):
        s.run(1, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s.mk.close()


@pytest.mark.parametrize("batch, beams, vocab, n_out", [(1, 4, 1000, 4), (2, 4, 128256, 8), (70, 3, 500, 6), (3, 16, 200, 32)])
def test_selection_behind_a_failed_step(batch, beams, vocab, n_out):
    logits = torch.randn(batch * beams, vocab, device="cuda")
    scores = torch.randn(batch, beams, device="cuda")
    fin = torch.zeros(batch, beams, dtype=torch.int32, device="cuda")

    def outputs():
        return ([torch.full((batch, n_out), 5, dtype=torch.int32, device="cuda") for _ in range(2)]
                + [torch.full((batch, n_out), 5.0, device="cuda"), torch.full((batch, n_out), 5, dtype=torch.int32, device="cuda"),
                   i32([3] * (batch * beams))])

    def choose(o, **kw):
        beam_select(logits, scores, o[0], o[1], o[2], finished=fin, eos=3, next_finished=o[3], positions=o[4], **kw)

    plain, status = outputs(), i32([0])
    choose(plain)
    got = outputs()
    choose(got, status=status)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(plain, got))
    for code in (BAD_POSITION, -1):
        status.fill_(code)
        got, was = outputs(), outputs()
        choose(got, status=status)
        torch.cuda.synchronize()
        assert torch.all(got[1] == -1)
        assert all(torch.equal(got[i], was[i]) for i in (0, 2, 3, 4))
    with pytest.raises(AssertionError, match="status"):
        choose(got, status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(AssertionError, match="status"):
        choose(got, status=0)


def test_a_captured_search_stops_when_a_replay_reaches_the_end():
    s, t = Search("8-bit"), Search("8-bit")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    par = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = s.mk.decode_step_qcache_workspace(s.cache, 4, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.mk.decode_steps_beam(s.tokens, s.positions, s.cache, s.logits, s.scores, 1, finished=s.finished, eos=7, starts=s.starts,
                               parents=par, workspace=ws, status=status)
    codes = []
    for _ in range(6):
        graph.replay()
        codes.append(int(status.item()))
    assert codes == [0] * 4 + [BAD_POSITION] * 2 and torch.all(par == -1)
    t.run(4)
    assert all(torch.equal(x, y) for x, y in zip(s.state(), t.state()))
    s.mk.close()
    t.mk.close()


@pytest.mark.parametrize("kind", ["8-bit", "bf16"])
def test_logits_of_a_larger_batch(kind):
    """A buffer with room for more rows than the step has (one for max_batch, say) gives the same search."""
    a, b = Search(kind, past=(10, 12)), Search(kind, past=(10, 12))
    b.logits = torch.full((7, TINY.vocab), 50.0, device="cuda")
    want, got = a.run(5), b.run(5)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    assert torch.equal(a.logits, b.logits[:4]) and torch.all(b.logits[4:] == 50)
    b.logits = b.logits[:3]
    with pytest.raises(AssertionError):
        b.run(1)
    a.mk.close()
    b.mk.close()
