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
