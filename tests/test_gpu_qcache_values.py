"""Attention over the 8-bit cache where values, scores and lengths are not the ordinary ones, against a 64-bit form that is
built from the appended tokens and the rows' own lengths (never read back from the cache).

Tolerance, relative to max |v|: a score is a sum of dim products of a whole number and a query held in 30 bits, added in
fp32, off by at most (dim + 8) 2^-23 of A = max_s sum_d |q_d k_sd| / sqrt(dim), and an exponent's argument by 2^-22 of its own
size (at most 2 A + 32); a weight moves by as much, an output by twice it, and the sums add (keys / 4 + 64) 2^-23. Value scales
of 2^-E .. 2^E enter the outputs' exponents and the factor behind them: three roundings of numbers of that size, 2^-22 E."""
import numpy as np
import pytest
import torch

from cases_beam_cache import BLOCK, attend, quantise
from persistent_megakernel_interpreter_b200.config import ModelConfig
from persistent_megakernel_interpreter_b200.qcache import QCache

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def stored(x):
    """The values (64-bit) that a row of tokens x [n][dim] is held as: closed blocks quantised, the open one as it is."""
    out = x.astype(np.float64)
    for i in range(len(x) // BLOCK):
        codes, scale = quantise(x[i * BLOCK:(i + 1) * BLOCK])
        out[i * BLOCK:(i + 1) * BLOCK] = codes.astype(np.float64) * np.float64(scale)
    return out


class Rows:
    """A cache of one layer filled with lengths[r] tokens of k, v [rows][heads][slots][dim] (bf16), and what it holds."""

    def __init__(self, k, v, lengths, max_seq=None):
        rows, heads, slots, dim = k.shape
        self.cfg = ModelConfig("shape", 1, 512, heads, heads, dim, 1024, 4096)
        self.cache = QCache(self.cfg, rows, max_seq or slots)
        self.cache.append(k[None].cuda(), v[None].cuda(), i32([0] * rows), counts=i32(lengths))
        self.lengths = list(lengths)
        self.k, self.v = ([[stored(t[r, h, :n].float().numpy()) for h in range(heads)] for r, n in enumerate(lengths)]
                          for t in (k, v))

    def check(self, q, positions, max_ctx, extra=0.0, keys=None, **kw):
        """keys[r]: the slots row r attends to (positions[r] + 1 where None)."""
        rows, n_heads, dim = q.shape
        heads = self.cfg.n_kv_heads
        out = torch.full((rows, n_heads, dim), 7.0, device="cuda")
        self.cache.attention(0, q.cuda(), i32(positions), out, max_ctx=max_ctx, **kw)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy().reshape(rows, heads, -1, dim)
        qn = q.double().numpy().reshape(rows, heads, -1, dim)
        for r in range(rows):
            n = positions[r] + 1 if keys is None else keys[r]
            for h in range(heads):
                k, v = self.k[r][h][:n], self.v[r][h][:n]
                if n == 0:
                    assert np.all(got[r, h] == 0)
                    continue
                ref = attend(qn[r, h], k, v)
                a = np.max(np.abs(qn[r, h]) @ np.abs(k).T) / np.sqrt(dim)
                big = np.max(np.abs(v))
                tol = (2 * ((dim + 8) * 2.0 ** -23 * a + 2.0 ** -22 * (2 * a + 32)) + (n / 4 + 64) * 2.0 ** -23 + extra) * big
                err = np.abs(got[r, h] - ref)
                assert np.all(err <= tol), (r, h, n, np.max(err) / big, tol / big)


def normal(g, *size):
    return torch.from_numpy(g.standard_normal(size).astype(np.float32))


# One CTA per row and head, and the split, with enough keys for several batches of a warp
SIZES = [(64, 640), (128, 512), (64, 200000), (128, 100000)]


@pytest.mark.parametrize("dim, n", SIZES)
@pytest.mark.parametrize("amp", [1.0, 1e-4, 1e-6, 1e-9])
def test_blocks_of_zero_values_ahead_of_small_ones(dim, n, amp):
    """A block of zeros has no scale; whatever a warp meets first must not set the size that weights are held relative to."""
    g = np.random.default_rng(int(n + dim))
    k, v = normal(g, 1, 1, n, dim), normal(g, 1, 1, n, dim) * amp
    zero = (np.arange(n) // BLOCK) % 16 < 8
    v[0, 0, zero] = 0
    rows = Rows(k.bfloat16(), v.bfloat16(), [n])
    rows.check(normal(g, 1, 3, dim), [n - 1], n, extra=2.0 ** -22 * 40)


@pytest.mark.parametrize("dim, n", SIZES)
@pytest.mark.parametrize("first, second", [(80, -58), (-58, 80), (60, -45)])
def test_values_of_sizes_far_apart(dim, n, first, second):
    """Blocks of 2^80 and of 2^-58 at equal scores: each key keeps its share of the softmax's sum."""
    g = np.random.default_rng(n + first)
    k, v = normal(g, 1, 1, n, dim) * 0.1, normal(g, 1, 1, n, dim)
    at = (np.arange(n) // BLOCK) % 16 < 8
    v[0, 0, at] *= 2.0 ** first
    v[0, 0, ~at] *= 2.0 ** second
    rows = Rows(k.bfloat16(), v.bfloat16(), [n])
    q = normal(g, 1, 4, dim)
    q[0, 0] = 0
    rows.check(q, [n - 1], n, extra=2.0 ** -22 * 100)


# ------------------------------------------------------------------ slots before a row's last

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads, group", [(2, 4), (3, 1)])
@pytest.mark.parametrize("lengths, cuts", [([1000, 992, 40, 650], [650, 641, 672, 1, 33, 991]),
                                           ([2500, 2496, 2490, 1100], [2489, 1999, 1025, 2496, 70])])
def test_max_ctx_cuts_rows_anywhere(dim, heads, group, lengths, cuts):
    """max_ctx inside closed blocks, inside the open one and at their borders, with rows that end before it."""
    g = np.random.default_rng(dim + heads)
    rows, slots = len(lengths), max(lengths)
    k, v = (normal(g, rows, heads, slots, dim).bfloat16() for _ in range(2))
    rows_ = Rows(k, v, lengths)
    for cut in cuts:
        q = normal(g, rows, heads * group, dim)
        rows_.check(q, [n - 1 for n in lengths], cut, keys=[min(n, cut) for n in lengths])
        rows_.check(q, [n - 1 for n in lengths], cut, keys=[min(n, cut) for n in lengths], lengths=i32(lengths))


def test_positions_far_beyond_max_ctx():
    """The largest position means a full cache, whose last block is open where max_seq is no multiple of 32."""
    g = np.random.default_rng(4)
    for max_seq, cuts in ((100, (100, 99, 96, 95, 33)), (2000, (2000, 1985, 1984, 1950, 1100))):
        k, v = (normal(g, 2, 2, max_seq, 64).bfloat16() for _ in range(2))
        rows = Rows(k, v, [max_seq, max_seq])
        for cut in cuts:
            rows.check(normal(g, 2, 4, 64), [2 ** 31 - 1, -2 ** 31], cut, keys=[cut, 0])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_seq", [300, 2300])
def test_any_slots_of_rows_of_known_lengths(dim, max_seq):
    """Every kind of prefix; positions and max_ctx beyond the length stop at it. What is not attended to may be anything."""
    g = np.random.default_rng(max_seq + dim)
    lengths = [max_seq, max_seq // 32 * 32, 257, 31, 0]
    k, v = (normal(g, 5, 2, max_seq, dim).bfloat16() for _ in range(2))
    k[:, :, 96:128] = 0                                      # a block of zero keys, some of them cut off
    rows = Rows(k, v, lengths)
    for tail in (rows.cache.k_tail, rows.cache.v_tail):
        for r, n in enumerate(lengths):
            tail[:, r, :, n % BLOCK:] = float("nan")
    for at in ([max_seq - 1] * 5, [250, 100, 255, 30, 0], [255, 96, 256, 0, -1], [0, 31, 32, 40, 7], [-1, 97, 257, -9, 2 ** 31 - 1],
               [126, 127, 128, 5, 5], [max_seq - 2, max_seq - 45, 224, 8, 0]):
        for max_ctx in (max_seq, max_seq - 37, 101):
            keys = [max(0, min(p + 1, n, max_ctx)) for p, n in zip(at, lengths)]
            q = normal(g, 5, 6, dim)
            rows.check(q, at, max_ctx, keys=keys, lengths=i32(lengths))
            q[:, :] = 0
            rows.check(q, at, max_ctx, keys=keys, lengths=i32(lengths))


def test_a_bad_block_behind_the_cut_is_not_seen():
    g = np.random.default_rng(5)
    for n, cut in ((320, 200), (2400, 2200)):
        k, v = (normal(g, 1, 1, n, 64) for _ in range(2))
        k[0, 0, cut // BLOCK * BLOCK + BLOCK] = float("nan")
        v[0, 0, cut // BLOCK * BLOCK + BLOCK + 1] = float("inf")
        rows = Rows(k.bfloat16(), v.bfloat16(), [cut // BLOCK * BLOCK + BLOCK])   # what is attended to, as it is held
        rows.cache.append(k[None].bfloat16().cuda(), v[None].bfloat16().cuda(), i32([0]))
        rows.check(normal(g, 1, 4, 64), [n - 1], cut, keys=[cut])
        rows.check(normal(g, 1, 4, 64), [cut - 1], n, keys=[cut], lengths=i32([n]))


def test_lengths_on_the_host_or_too_few_are_refused():
    cache = QCache(ModelConfig("shape", 1, 512, 1, 1, 64, 1024, 4096), 2, 64)
    q, out = torch.zeros(2, 4, 64, device="cuda"), torch.full((2, 4, 64), 7.0, device="cuda")
    for bad in (torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda"),
                torch.zeros(2, dtype=torch.int64, device="cuda")):
        with pytest.raises(AssertionError, match="lengths"):
            cache.attention(0, q, i32([0, 0]), out, lengths=bad)
    torch.cuda.synchronize()
    assert torch.all(out == 7)


# ------------------------------------------------------------------ scores far from the ordinary ones

def check_one_sided(dim, n, good, bad, query, seed):
    """Keys of one dim only, `good` for a third of them and `bad` for the others, and queries `query` there. A score x moves by up
    to 2^-22 |x| on its way to a weight, which beyond 2^22 says nothing of the good keys' shares any more; but the bad ones, a
    third of x away, have none. So an output is finite and lies among the good keys' values."""
    g = np.random.default_rng(seed)
    k, v = torch.zeros(1, 1, n, dim), normal(g, 1, 1, n, dim).bfloat16()
    best = g.permutation(n) < (n + 2) // 3
    k[0, 0, :, 0] = torch.from_numpy(np.where(best, good, bad).astype(np.float32))
    rows = Rows(k.bfloat16(), v, [n])
    q, out = torch.zeros(1, 4, dim), torch.empty(1, 4, dim, device="cuda")
    q[:, :, 0] = query
    rows.cache.attention(0, q.cuda(), i32([n - 1]), out)
    torch.cuda.synchronize()
    got, among = out[0].double().cpu().numpy(), rows.v[0][0][best]
    tol = (n / 4 + 64) * 2.0 ** -23 * np.abs(among).max()
    assert np.all(got >= among.min(0) - tol) and np.all(got <= among.max(0) + tol), query


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [20, 32, 640, 650, 2570])
@pytest.mark.parametrize("good, bad", [(-3.0, -5.0), (5.0, 3.0), (0.0, -3.0)])
def test_scores_far_from_zero(dim, n, good, bad):
    for query in (1e5, 1e8, 3e12, 1e20, 1e32, 1e36):
        check_one_sided(dim, n, good, bad, query, n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [20, 32, 640, 650, 2570])
def test_queries_of_the_largest_number(dim, n):
    """Any finite query counts: scores of 1e35 here."""
    for sign in (1.0, -1.0):
        check_one_sided(dim, n, sign * 2.0 ** -8, 0.0, sign * torch.finfo(torch.float32).max, n)


@pytest.mark.parametrize("max_ctx", [900, 2000])
def test_prefixes_captured_and_replayed_with_other_lengths(max_ctx):
    g = np.random.default_rng(max_ctx)
    k, v = (normal(g, 2, 2, 2000, 64).bfloat16() for _ in range(2))
    rows = Rows(k, v, [2000, 1500])
    q = normal(g, 2, 8, 64)
    qd, out = q.cuda(), torch.zeros(2, 8, 64, device="cuda")
    pos, lengths, ws = i32([0, 0]), i32([2000, 1500]), rows.cache.attention_workspace(2, 8, max_ctx)
    rows.cache.attention(0, qd, pos, out, max_ctx=max_ctx, workspace=ws, lengths=lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows.cache.attention(0, qd, pos, out, max_ctx=max_ctx, workspace=ws, lengths=lengths)
    for at in ([1999, 1499], [40, 1000], [-1, 70], [899, 3]):
        pos.copy_(i32(at))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        rows.check(q, at, max_ctx, keys=[min(p + 1, max_ctx) for p in at], lengths=lengths)
        rows.cache.attention(0, qd, pos, out, max_ctx=max_ctx, workspace=ws, lengths=lengths)
        torch.cuda.synchronize()
        assert torch.equal(got, out)
