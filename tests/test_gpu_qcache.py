"""The 8-bit cache on the GPU: stored blocks and reordering are exact; attention against a 64-bit form.

Attention's tolerance, from its arithmetic. A score is a sum of dim products of a whole number and a query held in 22
bits, added in fp32: off by at most (dim + 8) 2^-23 of A = max_s sum_d |q_d k_sd| / sqrt(dim), and the exponent's argument
by 2^-22 of its own size (at most 2 A + 32). That moves a weight by the same relative amount, an output by twice it, and
the output's own sum adds (keys / 4 + 64) 2^-23: all of that of max |v|."""
import numpy as np
import pytest
import torch

from cases_beam_cache import BLOCK, attend, quantise, reorder
from persistent_megakernel_interpreter_b200.config import ModelConfig, TINY
from persistent_megakernel_interpreter_b200.inputs import make_kv_cache, make_tokens, make_weights
from persistent_megakernel_interpreter_b200.model import Megakernel
from persistent_megakernel_interpreter_b200.qcache import QCache

pytestmark = pytest.mark.gpu


def shape(layers, heads, dim):
    return ModelConfig("shape", layers, 512, heads, heads, dim, 1024, 4096)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def bf16(g, *size, scale=1.0):
    return (torch.from_numpy(g.standard_normal(size).astype(np.float32)) * scale).to(torch.bfloat16)


class Model:
    """What a cache holds, kept on the host: every token of every row in bf16."""

    def __init__(self, layers, rows, heads, dim, max_seq):
        self.kv = [np.zeros((layers, rows, heads, max_seq, dim), np.float32) for _ in range(2)]
        self.n = np.zeros(rows, int)

    def expect(self, which, l, r, h):
        """codes, scales and open tokens of one row and head."""
        x = self.kv[which][l, r, h, :self.n[r]]
        nb = len(x) // BLOCK
        parts = [quantise(x[i * BLOCK:(i + 1) * BLOCK]) for i in range(nb)]
        return parts, x[nb * BLOCK:]


def check_cache(c, m, rows=None):
    codes = [c.k_codes.cpu().numpy(), c.v_codes.cpu().numpy()]
    scales = [c.k_scale.cpu().numpy(), c.v_scale.cpu().numpy()]
    tails = [c.k_tail.float().cpu().numpy(), c.v_tail.float().cpu().numpy()]
    layers, all_rows, heads = codes[0].shape[:3]
    for w in range(2):
        for l in range(layers):
            for r in range(all_rows if rows is None else rows):
                for h in range(heads):
                    parts, rest = m.expect(w, l, r, h)
                    for i, (code, scale) in enumerate(parts):
                        got = scales[w][l, r, h, i]
                        assert (np.isnan(scale) and np.isnan(got)) or got == scale
                        if code is not None:
                            assert np.array_equal(codes[w][l, r, h, i * BLOCK:(i + 1) * BLOCK], code)
                    assert np.array_equal(tails[w][l, r, h, :len(rest)], rest)


def give(c, m, g, counts, first_layer=0, layers=None, order=(0, 1, 2, 3), scale=1.0, n_new=None):
    """Appends counts[r] random tokens to each row of both; `order`: how the source is laid out in memory."""
    layers = c.n_layers - first_layer if layers is None else layers
    rows, n = len(counts), n_new or max(max(counts), 1)
    size = (layers, rows, c.n_kv_heads, n)
    new = []
    for w in range(2):
        x = bf16(g, *(size[i] for i in order), c.head_dim, scale=scale)
        back = [order.index(i) for i in range(4)] + [4]
        new.append(x.cuda().permute(back))
        for r, k in enumerate(counts):
            if k:
                m.kv[w][first_layer:first_layer + layers, r, :, m.n[r]:m.n[r] + k] = x.permute(back)[:, r, :, :k].float().numpy()
    c.append(new[0], new[1], i32(m.n[:rows]), counts=i32(counts), first_layer=first_layer)
    torch.cuda.synchronize()


@pytest.mark.parametrize("layers, rows, heads, dim, max_seq", [(1, 1, 1, 64, 100), (2, 3, 2, 128, 300), (3, 8, 1, 64, 257),
                                                               (1, 2, 8, 128, 96)])
def test_append_piece_by_piece(layers, rows, heads, dim, max_seq):
    """Pieces of every kind of length: inside the open block, up to its end, over several blocks, none."""
    g = np.random.default_rng(dim + rows)
    c, m = QCache(shape(layers, heads, dim), rows, max_seq), Model(layers, rows, heads, dim, max_seq)
    untouched = c.k_codes.clone()
    for step in range(9):
        room = max_seq - m.n
        most = [1, 1, 31, 1, 33, 2, 64, 95, 7][step]
        counts = np.minimum(room, g.integers(0 if step else 1, most + 1, rows) if rows > 1 else most)
        give(c, m, g, counts.tolist(), order=[(0, 1, 2, 3), (3, 1, 0, 2), (1, 3, 0, 2)][step % 3])
        m.n[:rows] += counts
        check_cache(c, m)
    closed = m.n // BLOCK * BLOCK
    for r in range(rows):                                    # slots of blocks that are not closed were not written
        assert torch.equal(c.k_codes[:, r, :, closed[r]:], untouched[:, r, :, closed[r]:])


def test_append_takes_over_a_bf16_cache_and_single_layers():
    g = np.random.default_rng(8)
    cfg = shape(3, 2, 64)
    k, v = make_kv_cache(cfg, 4, 200, past=[200, 0, 33, 64], seed=3)
    c, m = QCache(cfg, 4, 200), Model(3, 4, 2, 64, 200)
    c.append(k.cuda(), v.cuda(), i32([0] * 4), counts=i32([200, 0, 33, 64]))
    m.kv, m.n = [k.float().numpy().copy(), v.float().numpy().copy()], np.array([200, 0, 33, 64])
    check_cache(c, m)
    # one decoded token of two rows, layer by layer
    m.n = np.array([199, 0, 33, 64])
    for layer in range(3):
        give(c, m, g, [0, 1], first_layer=layer, layers=1)
    m.n[1] = 1
    check_cache(c, m)


def test_rows_that_cannot_be_appended_are_left():
    g = np.random.default_rng(9)
    c, m = QCache(shape(1, 1, 64), 6, 64), Model(1, 6, 1, 64, 64)
    give(c, m, g, [60, 40, 3, 3, 3, 3])
    m.n = np.array([60, 40, 3, 3, 3, 3])
    before = [t.clone() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail)]
    x = bf16(g, 1, 6, 1, 5, 64).cuda()
    # past the end, before the start, negative and too large counts, a position far out
    c.append(x, x, i32([60, -1, 3, 3, 2 ** 31 - 3, 64]), counts=i32([5, 2, -1, 6, 4, 1]))
    torch.cuda.synchronize()
    for old, new in zip(before, (c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail)):
        assert torch.equal(old, new)


def test_blocks_of_zeros_tiny_values_and_bad_numbers():
    c = QCache(shape(1, 1, 64), 1, 320)
    x = torch.zeros(1, 1, 1, 192, 64, dtype=torch.bfloat16)
    x[0, 0, 0, 40, 3] = 1e-30                                # tiny: held as zeros
    x[0, 0, 0, 70, 5] = float("inf")
    x[0, 0, 0, 100, 0] = float("nan")
    x[0, 0, 0, 130, 0] = -3.3e38
    x[0, 0, 0, 161, 1] = 2.0 ** -60
    c.append(x.cuda(), x.cuda(), i32([0]))
    torch.cuda.synchronize()
    m = Model(1, 1, 1, 64, 320)
    m.kv, m.n = [x.float().numpy()] * 2, np.array([192])
    check_cache(c, m)
    assert torch.all(c.k_codes[0, 0, 0, :64] == 0) and torch.equal(c.k_scale[0, 0, 0, :2], torch.zeros(2, device="cuda"))


# ------------------------------------------------------------------ attention

def held(c, layer, row, head, n):
    """The values the cache holds, in 64 bits."""
    out = []
    for codes, scale, tail in ((c.k_codes, c.k_scale, c.k_tail), (c.v_codes, c.v_scale, c.v_tail)):
        nb = n // BLOCK
        x = codes[layer, row, head, :nb * BLOCK].double() * scale[layer, row, head, :nb].double().repeat_interleave(BLOCK)[:, None]
        out.append(torch.cat([x, tail[layer, row, head, :n - nb * BLOCK].double()]).cpu().numpy())
    return out


def check_attention(c, layer, q, positions, max_ctx, workspace=None):
    rows, n_heads, dim = q.shape
    out = torch.full((rows + 1, n_heads, dim), 7.0, device="cuda")
    c.attention(layer, q, i32(positions), out[:rows], max_ctx=max_ctx, workspace=workspace)
    torch.cuda.synchronize()
    assert torch.all(out[rows] == 7)                         # behind the last row
    group = n_heads // c.n_kv_heads
    got = out[:rows].double().cpu().numpy().reshape(rows, c.n_kv_heads, group, dim)
    qn = q.double().cpu().numpy().reshape(rows, c.n_kv_heads, group, dim)
    for r in range(rows):
        n = min(max(positions[r] + 1, 0), max_ctx)
        for h in range(c.n_kv_heads):
            k, v = held(c, layer, r, h, n)
            ref = attend(qn[r, h], k, v)
            if n == 0:
                assert np.all(got[r, h] == 0)
                continue
            a = np.max(np.abs(qn[r, h]) @ np.abs(k).T) / np.sqrt(dim)
            tol = (2 * ((dim + 8) * 2.0 ** -23 * a + 2.0 ** -22 * (2 * a + 32)) + (n / 4 + 64) * 2.0 ** -23) * np.max(np.abs(v))
            assert np.all(np.abs(got[r, h] - ref) <= tol), (r, h, n, np.max(np.abs(got[r, h] - ref)), tol)


def filled(layers, rows, heads, dim, max_seq, lengths, seed, scale=1.0):
    g = np.random.default_rng(seed)
    c = QCache(shape(layers, heads, dim), rows, max_seq)
    x = [bf16(g, layers, rows, heads, max_seq, dim, scale=scale).cuda() for _ in range(2)]
    x[0][:, :, :, 0] *= 4                                    # a token that draws much of the weight
    c.append(x[0], x[1], i32([0] * rows), counts=i32(lengths))
    return c, g


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads, group", [(1, 1), (2, 3), (8, 4), (3, 2)])
@pytest.mark.parametrize("max_seq, lengths", [(32, [1, 31, 32]), (130, [129, 64, 0, 33]), (512, [512, 511, 96, 1, 0, 7, 33, 480]),
                                             (700, [700]), (2100, [2083, 0, 1, 1024, 64])])
def test_attention_against_the_64_bit_form(dim, heads, group, max_seq, lengths):
    rows = len(lengths)
    c, g = filled(2, rows, heads, dim, max_seq, lengths, dim + max_seq + group)
    q = torch.from_numpy(g.standard_normal((rows, heads * group, dim)).astype(np.float32) * 2).cuda()
    for layer in range(2):
        check_attention(c, layer, q, [n - 1 for n in lengths], max_seq)


@pytest.mark.parametrize("dim, heads, rows, n", [(64, 8, 2, 16384), (128, 2, 1, 40001), (64, 1, 1, 70000)])
def test_attention_over_long_contexts(dim, heads, rows, n):
    c, g = filled(1, rows, heads, dim, n, [n - 37 * r for r in range(rows)], n)
    q = torch.from_numpy(g.standard_normal((rows, 4 * heads, dim)).astype(np.float32)).cuda()
    check_attention(c, 0, q, [n - 1 - 37 * r for r in range(rows)], n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows, heads, group", [(1, 1, 1), (3, 1, 3), (1, 5, 1), (5, 7, 2)])
def test_attention_on_either_side_of_its_two_forms(dim, rows, heads, group):
    """Contexts at the border between one CTA per pair and the split, and one past it; odd numbers of partials."""
    for max_ctx in (65536 // dim, 65536 // dim + 1, 131072 // dim, 131072 // dim + 1):
        lengths = [max(0, max_ctx - 31 * r - r * r) for r in range(rows)]
        c, g = filled(1, rows, heads, dim, max_ctx, lengths, max_ctx + rows)
        q = torch.from_numpy(g.standard_normal((rows, heads * group, dim)).astype(np.float32)).cuda()
        check_attention(c, 0, q, [n - 1 for n in lengths], max_ctx)


@pytest.mark.parametrize("max_ctx", [100, 5000])
def test_rows_that_are_all_empty(max_ctx):
    c = QCache(shape(1, 2, 64), 3, max_ctx)
    q, out = torch.randn(3, 4, 64, device="cuda"), torch.full((3, 4, 64), 7.0, device="cuda")
    c.attention(0, q, i32([-1, -2 ** 31, -7]), out)
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_positions_written_by_the_kernel_just_before():
    """The attention's kernels are placed while the one before them ends; what that one wrote has to be seen."""
    for max_ctx in (400, 4000):
        c, g = filled(1, 2, 2, 64, max_ctx, [max_ctx, max_ctx], 31)
        q = torch.from_numpy(g.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
        at = [i32([max_ctx - 1, 40]), i32([33, max_ctx // 2]), i32([max_ctx // 3, -1])]
        ws = c.attention_workspace(2, 4, max_ctx)
        want = []
        for p in at:
            out = torch.empty(2, 4, 64, device="cuda")
            c.attention(0, q, p, out, workspace=ws)
            torch.cuda.synchronize()
            want.append(out)
        pos, q2 = at[0].clone(), q.clone()
        outs = [torch.empty(2, 4, 64, device="cuda") for _ in range(300)]
        for i, out in enumerate(outs):
            q2.zero_()
            q2.copy_(q)
            pos.copy_(at[i % 3])
            c.attention(0, q2, pos, out, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(out, want[i % 3]) for i, out in enumerate(outs))


def test_attention_reads_no_slot_behind_the_last():
    """Garbage (NaN scales, tails of NaN) behind each row's length, and a position beyond max_ctx."""
    lengths = [70, 64, 33, 0]
    for max_seq in (200, 1500):
        c, g = filled(1, 4, 2, 64, max_seq, lengths, 5)
        for r, n in enumerate(lengths):
            for scale, tail in ((c.k_scale, c.k_tail), (c.v_scale, c.v_tail)):
                scale[:, r, :, n // BLOCK:] = float("nan")
                tail[:, r, :, n % BLOCK:] = float("nan")
        q = torch.from_numpy(g.standard_normal((4, 8, 64)).astype(np.float32)).cuda()
        check_attention(c, 0, q, [n - 1 for n in lengths], max_seq)
    c, g = filled(1, 2, 2, 64, 1000, [1000, 1000], 6)
    q = torch.from_numpy(g.standard_normal((2, 8, 64)).astype(np.float32)).cuda()
    check_attention(c, 0, q, [10 ** 6, 640 - 1], 640)        # closed blocks only
    check_attention(c, 0, q, [2 ** 31 - 1, -5], 640)


@pytest.mark.parametrize("max_seq", [320, 1920])
def test_attention_with_blocks_of_zeros_and_of_very_different_scales(max_seq):
    rows, g = 3, np.random.default_rng(7)
    c = QCache(shape(1, 2, 64), rows, max_seq)
    k, v = (bf16(g, 1, rows, 2, max_seq, 64) for _ in range(2))
    v[:, 0, :, 32:96] = 0                                    # zero values between others
    v[:, 1, :, :64] = 0                                      # at the start
    k[:, 1, :, 96:128] = 0                                   # zero keys
    v[:, 2, :, 64:128] *= 1e-6
    v[:, 2, :, 128:160] *= 1e4
    c.append(k.cuda(), v.cuda(), i32([0] * rows))
    q = torch.from_numpy(g.standard_normal((rows, 6, 64)).astype(np.float32)).cuda()
    for n in (max_seq, 64, 33, 96):
        check_attention(c, 0, q, [n - 1] * rows, max_seq)
    c.append(torch.zeros_like(k).cuda(), torch.zeros_like(v).cuda(), i32([0] * rows))
    out = torch.full((rows, 6, 64), 7.0, device="cuda")
    c.attention(0, q, i32([max_seq - 1] * rows), out)
    assert torch.all(out == 0)


@pytest.mark.parametrize("scale", [1e-20, 1e6])
def test_queries_of_any_size(scale):
    c, g = filled(1, 2, 2, 64, 1600, [1600, 90], 12, scale=1 / scale if scale > 1 else 1.0)
    q = torch.from_numpy(g.standard_normal((2, 8, 64)).astype(np.float32) * np.float32(scale)).cuda()
    check_attention(c, 0, q, [1599, 89], 1600)
    check_attention(c, 0, torch.zeros_like(q), [599, 89], 600)


@pytest.mark.parametrize("max_seq", [300, 1900])
def test_a_bad_block_gives_nan_and_only_to_its_row_and_head(max_seq):
    g = np.random.default_rng(13)
    c = QCache(shape(1, 2, 64), 2, max_seq)
    k, v = (bf16(g, 1, 2, 2, max_seq, 64) for _ in range(2))
    k[0, 0, 1, 40, 5] = float("inf")
    v[0, 1, 0, 70, 5] = float("nan")
    c.append(k.cuda(), v.cuda(), i32([0, 0]))
    q = torch.from_numpy(g.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
    out = torch.zeros(2, 4, 64, device="cuda")
    c.attention(0, q, i32([max_seq - 1] * 2), out)
    nan = torch.isnan(out).reshape(2, 2, 2 * 64).all(2).cpu().numpy()
    some = torch.isnan(out).reshape(2, 2, 2 * 64).any(2).cpu().numpy()
    assert np.array_equal(nan, [[False, True], [True, False]]) and np.array_equal(some, nan)


def test_attention_captured_replayed_and_on_other_streams():
    c, g = filled(1, 2, 2, 64, 3000, [3000, 1500], 14)
    q = torch.from_numpy(g.standard_normal((2, 8, 64)).astype(np.float32)).cuda()
    pos, out = i32([2999, 1499]), torch.zeros(2, 8, 64, device="cuda")
    c.attention(0, q, pos, out)
    torch.cuda.synchronize()
    want = out.clone()
    for ws in (None, c.attention_workspace(2, 8, 3000)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.attention(0, q, pos, out, workspace=ws)
        for _ in range(3):
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    outs, streams = [torch.zeros_like(out) for _ in range(6)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        c.attention(0, q, pos, o, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("layers, rows, heads, dim, max_seq", [(2, 4, 2, 64, 300), (1, 8, 1, 128, 96), (3, 3, 5, 64, 1000)])
def test_qcache_reorder_against_the_plain_form(layers, rows, heads, dim, max_seq):
    g = np.random.default_rng(max_seq)
    for trial in range(5):
        lengths = g.integers(0, max_seq + 1, rows)
        c, _ = filled(layers, rows, heads, dim, max_seq, np.maximum(lengths, 0).tolist(), trial)
        parents = g.integers(-1, rows, rows)
        starts = None if trial == 0 else g.integers(0, max_seq + 1, rows)
        old = [t.clone() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail)]
        c.reorder(i32(parents), i32(lengths), starts=None if starts is None else i32(starts))
        torch.cuda.synchronize()
        s = np.zeros(rows, int) if starts is None else starts
        spans = [lambda p, r: (s[r] // BLOCK * BLOCK, lengths[p] // BLOCK * BLOCK)] * 2 + \
                [lambda p, r: (s[r] // BLOCK, lengths[p] // BLOCK)] * 2 + \
                [lambda p, r: (max(0, s[r] - lengths[p] // BLOCK * BLOCK), lengths[p] % BLOCK)] * 2
        now = (c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail)
        for got, was, span in zip(now, old, spans):
            view = torch.int16 if got.dtype == torch.bfloat16 else torch.int32 if got.dtype == torch.float32 else torch.int8
            assert np.array_equal(got.view(view).cpu().numpy(), reorder(was.view(view).cpu().numpy(), parents, span))


def test_a_cache_beyond_32_bit_offsets():
    """More than 2^32 bytes of codes: the last layer's last planes are stored, attended to and reordered."""
    g = np.random.default_rng(3)
    max_seq = 1 << 20
    c = QCache(shape(3, 6, 128), 2, max_seq)
    x = [bf16(g, 1, 2, 6, 100, 128).cuda() for _ in range(2)]
    c.append(x[0], x[1], i32([0, 0]), counts=i32([100, 77]), first_layer=2)
    c.append(x[0][:, :, :, :64], x[1][:, :, :, :64], i32([max_seq, max_seq - 64]), first_layer=2)  # one does not fit
    torch.cuda.synchronize()
    for t, codes, scale in ((x[0], c.k_codes, c.k_scale), (x[1], c.v_codes, c.v_scale)):
        want, big = quantise(t[0, 1, 5, 32:64].float().cpu().numpy())
        assert np.array_equal(codes[2, 1, 5, -32:].cpu().numpy(), want) and float(scale[2, 1, 5, -1]) == big
        assert not codes[2, 0, 5, -64:].any()
    assert not c.k_codes[:2].any() and not c.v_codes[:2].any()
    q = torch.from_numpy(g.standard_normal((2, 12, 128)).astype(np.float32)).cuda()
    check_attention(c, 2, q, [99, 76], max_seq)
    check_attention(c, 2, q, [99, 76], 128)
    k0, v0, t0 = c.k_codes[2, 0].clone(), c.v_codes[2, 1].clone(), c.k_tail[2].clone()
    c.reorder(i32([1, 0]), i32([100, 77]))
    torch.cuda.synchronize()
    assert torch.equal(c.k_codes[2, 1, :, :96], k0[:, :96]) and torch.equal(c.v_codes[2, 0, :, :64], v0[:, :64])
    assert torch.equal(c.k_tail[2, 0, :, :13], t0[1, :, :13]) and torch.equal(c.k_tail[2, 1, :, :4], t0[0, :, :4])


def test_tensors_on_the_host_are_refused():
    c = QCache(shape(1, 1, 64), 1, 64)
    x, q = torch.zeros(1, 1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 64)
    with pytest.raises(AssertionError):
        c.append(x, x, i32([0]))
    with pytest.raises(AssertionError):
        c.attention(0, q, i32([0]), q.cuda())
    with pytest.raises(AssertionError):
        c.attention(0, q.cuda(), torch.zeros(1, dtype=torch.int32), q.cuda())
    with pytest.raises(AssertionError):
        c.attention(0, q.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), q.cuda())
    with pytest.raises(AssertionError):
        c.reorder(i32([0]), torch.zeros(1, dtype=torch.int32))
    assert not c.k_tail.any()


# ------------------------------------------------------------------ decode steps on it

@pytest.mark.parametrize("batch, past", [(1, 5), (3, 28), (2, 130)])
def test_decode_steps_on_the_8_bit_cache(batch, past):
    """Against the same steps on a bf16 cache that holds what the 8-bit cache holds, block by block. The 8-bit values
    reach the bf16 cache rounded (2^-9), so logits agree to the decode step's pass line, 1e-2 of their largest; while
    nothing is quantised yet (fewer than 32 tokens) they agree to fp32 summation, 2^-7 / keys + 1e-4."""
    steps, max_seq = 8, 600
    w = make_weights(TINY, seed=1)
    mk = Megakernel(TINY, w.to("cuda"), max_batch=batch, max_seq=max_seq)
    k, v = make_kv_cache(TINY, batch, max_seq, past=past, seed=2)
    mk.build_schedule(batch, max_seq)
    for max_ctx in (max_seq, past + steps):
        c = QCache(TINY, batch, max_seq)
        c.append(k.cuda(), v.cuda(), i32([0] * batch), counts=i32([past] * batch))
        status, logits = torch.full((1,), 9, dtype=torch.int32, device="cuda"), torch.empty(batch, TINY.vocab, device="cuda")
        ref = torch.empty_like(logits)
        for i in range(steps):
            tok = make_tokens(TINY, batch, seed=20 + i).to(torch.int32).cuda()
            pos = i32([past + i] * batch)
            kd, vd = torch.zeros_like(k, device="cuda"), torch.zeros_like(v, device="cuda")
            n = past + i
            tails = c.k_tail.clone()
            mk.decode_step_qcache(tok, pos, c, logits, max_ctx=max_ctx, status=status)
            # what the step attended to, but for its own token: the block that it closed is quantised already
            nb = (n + 1) // BLOCK * BLOCK
            for to, codes, scale, tail in ((kd, c.k_codes, c.k_scale, c.k_tail), (vd, c.v_codes, c.v_scale, c.v_tail)):
                to[:, :, :, :nb] = (codes.float() * scale.repeat_interleave(BLOCK, 3)[:, :, :, :max_seq, None])[:, :, :, :nb]
                to[:, :, :, nb:n] = tail[:, :, :, :max(n - nb, 0)]
            mk.baseline_decode_step(tok, pos, kd, vd, ref)  # the same matrix products, on the CUDA cores
            torch.cuda.synchronize()
            assert int(status.item()) == 0 and mk.status()[0] == 0
            top = ref.abs().amax(1, keepdim=True)
            bar = 1e-2 if n + 1 >= BLOCK else 2.0 ** -7 / (n + 1) + 1e-4
            assert torch.all((logits - ref).abs() <= bar * top), (i, float(((logits - ref).abs() / top).max()))
            if (n + 1) % BLOCK:                              # the new key, layer 0: the same bits
                assert torch.equal(c.k_tail[0, :, :, n % BLOCK], kd[0, :, :, n])
                assert torch.equal(c.k_tail[:, :, :, :n % BLOCK], tails[:, :, :, :n % BLOCK])
            else:
                codes, scale = quantise(torch.cat([tails[0, 0, 0, :BLOCK - 1], kd[0, 0, 0, n:n + 1]]).float().cpu().numpy())
                assert np.array_equal(c.k_codes[0, 0, 0, n + 1 - BLOCK:n + 1].cpu().numpy(), codes)
                assert float(c.k_scale[0, 0, 0, n // BLOCK]) == scale
    mk.close()


def test_a_bad_step_stores_nothing():
    mk = Megakernel(TINY, make_weights(TINY, seed=1).to("cuda"), max_batch=2, max_seq=100)
    c = QCache(TINY, 2, 100)
    logits, status = torch.empty(2, TINY.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = mk.decode_step_qcache_workspace(c, 2, 100)
    ws.fill_(0xff)
    for tok, pos, code in (([1, TINY.vocab], [3, 3], 6), ([-1, 1], [3, 3], 6), ([1, 1], [3, 100], 7), ([1, 1], [-1, 3], 7)):
        mk.decode_step_qcache(i32(tok), i32(pos), c, logits, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == code
        assert not c.k_tail.any() and not c.v_tail.any() and not c.k_codes.any()
    mk.decode_step_qcache(i32([1, 2]), i32([0, 3]), c, logits, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and bool(c.k_tail.any()) and torch.isfinite(logits).all()
    assert mk.status()[0] == 0
    mk.close()


def test_steps_of_two_handles_of_different_batches():
    """The matvec kernels' shared-memory limit belongs to the kernel: a small handle's schedule does not lower it."""
    w = make_weights(TINY, seed=1).to("cuda")
    big, small = Megakernel(TINY, w, max_batch=8, max_seq=64), Megakernel(TINY, w, max_batch=1, max_seq=64)
    c = QCache(TINY, 8, 64)
    big.build_schedule(8, 64)
    small.build_schedule(1, 64)
    logits = torch.empty(8, TINY.vocab, device="cuda")
    kd = torch.zeros(2, 8, 2, 64, 64, dtype=torch.bfloat16, device="cuda")
    big.baseline_decode_step(i32(range(8)), i32([0] * 8), kd, kd.clone(), logits)
    want = logits.clone()
    big.decode_step_qcache(i32(range(8)), i32([0] * 8), c, logits)
    torch.cuda.synchronize()
    assert big.status()[0] == 0
    assert torch.allclose(logits, want, rtol=0, atol=float(1e-4 * want.abs().max()))
    big.close()
    small.close()


def test_beam_search_on_the_8_bit_cache():
    """decode_steps_beam on an 8-bit cache against its own steps, choices and reorders called one by one."""
    rows, beams, steps, past, max_seq = 6, 3, 9, 27, 96
    mk = Megakernel(TINY, make_weights(TINY, seed=3).to("cuda"), max_batch=rows, max_seq=max_seq)
    k, v = make_kv_cache(TINY, rows, max_seq, past=past, seed=4)
    for t in (k, v):
        for r in range(rows):
            t[:, r] = t[:, r // beams * beams]
    runs = []
    for one_call in (True, False):
        c = QCache(TINY, rows, max_seq)
        c.append(k.cuda(), v.cuda(), i32([0] * rows), counts=i32([past] * rows))
        tok = make_tokens(TINY, 2, seed=5).repeat_interleave(beams).to(torch.int32).cuda()
        pos, start = i32([past] * rows), i32([past] * rows)
        sc = torch.full((2, beams), -float("inf"), device="cuda")
        sc[:, 0] = 0
        lg = torch.empty(rows, TINY.vocab, device="cuda")
        gen, par = (torch.zeros(steps, rows, dtype=torch.int32, device="cuda") for _ in range(2))
        for i in range(1 if one_call else steps):
            n = steps if one_call else 1
            mk.decode_steps_beam(tok, pos, c, lg, sc, n, starts=start, generated=gen[i:], parents=par[i:])
        torch.cuda.synchronize()
        runs.append([t.cpu() for t in (gen, par, sc, pos, c.k_codes, c.v_codes, c.k_scale, c.k_tail, c.v_tail)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    gen, par = runs[0][:2]
    # each surviving row's history: following the parents back gives one token per step, all rows distinct
    texts = set()
    for r in range(rows):
        at, text = r, []
        for i in reversed(range(steps)):
            text.append(int(gen[i, at]))
            at = int(par[i, at])
        assert at // beams == r // beams
        texts.add((r // beams, tuple(text)))
    assert len(texts) == rows
    mk.close()


def test_beam_steps_captured_and_replayed():
    """A step, the choice and the reorder on the 8-bit cache in one graph, replayed, against the same calls."""
    rows, beams, steps, past, max_seq = 4, 2, 6, 29, 4000
    mk = Megakernel(TINY, make_weights(TINY, seed=3).to("cuda"), max_batch=rows, max_seq=max_seq)
    k, v = make_kv_cache(TINY, rows, 64, past=past, seed=4)
    ends = []
    for captured in (False, True):
        c = QCache(TINY, rows, max_seq)
        c.append(k.cuda(), v.cuda(), i32([0] * rows), counts=i32([past] * rows))
        tok = make_tokens(TINY, rows, seed=5).to(torch.int32).cuda()
        pos, start = i32([past] * rows), i32([past] * rows)
        sc = torch.zeros(2, beams, device="cuda")
        fin = torch.zeros(2, beams, dtype=torch.int32, device="cuda")
        lg = torch.empty(rows, TINY.vocab, device="cuda")
        ws = mk.decode_step_qcache_workspace(c, rows, max_seq)
        par = torch.zeros(rows, dtype=torch.int32, device="cuda")

        def step():
            mk.decode_steps_beam(tok, pos, c, lg, sc, 1, finished=fin, eos=7, starts=start, parents=par, workspace=ws)

        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            step = graph.replay
        for _ in range(steps):
            step()
        torch.cuda.synchronize()
        ends.append([t.cpu() for t in (tok, pos, sc, fin, par, lg, c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail)])
    assert all(torch.equal(a, b) for a, b in zip(*ends))
    mk.close()
