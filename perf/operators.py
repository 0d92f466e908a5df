"""Timed cases of the operators around a decode step: beam selection, cache reordering, and the 8-bit cache.

Four operators, named by a case's "op":

* ``select``: beam search's choice. Of the ``beams`` rows of logits of each sequence, the ``n_out`` best
  continuations by running score plus log-softmax. Order: larger total first, equal totals to the lower beam, within
  a beam the larger logit, equal logits the lower token. A finished beam offers ``eos`` at its own score only.
* ``reorder``: row r of a slot cache becomes row parents[r], slots starts[r] .. lengths[parents[r]] - 1, all rows at
  once and in place; of the bf16 cache (``bits`` 16) or of the 8-bit one (``bits`` 8).
* ``append``: new keys and values into an 8-bit cache: blocks of 32 tokens of one head hold codes
  rint(x * (127 / amax)) and the scale amax / 127; the tokens of the open block stay bf16 until it is full.
* ``attend``: one query token per row over that cache: softmax(q k / sqrt(dim)) v over slots 0 .. positions[row].

``run`` gives each in elementary torch operations, or (where ``own`` is true) by the framework's entry points.
Codes are int8 numbers and are returned as such, with their scales beside them: they have to be equal.
"""
import math

import numpy as np
import torch

own = False

T = 32  # tokens of a block of the 8-bit cache
NO_BLOCK = 2.0 ** -60  # a block whose largest magnitude is below this is held as zeros


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four beams of a small vocabulary, one sequence: the call's own latency
        {"name": "select 1x4 of 4096", "op": "select", "batch": 1, "beams": 4, "vocab": 4096, "n_out": 4, "done": 0},
        # a full batch of the decode step on the 1B vocabulary, twice as many candidates as beams, a finished beam
        {"name": "select 2x4 of 128256", "op": "select", "batch": 2, "beams": 4, "vocab": 128256, "n_out": 8, "done": 1},
        # many sequences over an odd vocabulary, rows off a 16-byte boundary
        {"name": "select 32x8 of 50257", "op": "select", "batch": 32, "beams": 8, "vocab": 50257, "n_out": 8, "done": 2},
        # the 2-layer model's cache, four beams, a short text
        {"name": "reorder tiny 4 rows", "op": "reorder", "bits": 16, "layers": 2, "heads": 2, "dim": 64, "seqs": 1, "beams": 4,
         "max_seq": 160, "length": 131, "start": 0},
        # the 1B cache, two sequences of four beams behind a shared prompt
        {"name": "reorder 1B 8 rows", "op": "reorder", "bits": 16, "layers": 16, "heads": 8, "dim": 64, "seqs": 2, "beams": 4,
         "max_seq": 4096, "length": 3777, "start": 512},
        # the same in 8 bits with 128-wide heads, all of a long text forked
        {"name": "reorder 8-bit 128-wide", "op": "reorder", "bits": 8, "layers": 28, "heads": 8, "dim": 128, "seqs": 1, "beams": 5,
         "max_seq": 8192, "length": 6001, "start": 0},
        # one decoded token of eight sequences, one layer
        {"name": "append 1 token", "op": "append", "layers": 1, "rows": 8, "heads": 8, "dim": 64, "tokens": 1, "past": 1000, "max_seq": 2048},
        # a prompt of every layer of the 1B model, ragged over four sequences
        {"name": "append 1B prompts", "op": "append", "layers": 16, "rows": 4, "heads": 8, "dim": 64, "tokens": 4001, "past": 0, "max_seq": 4352},
        # a long piece of one layer with 128-wide heads behind an open block
        {"name": "append 128-wide piece", "op": "append", "layers": 1, "rows": 2, "heads": 8, "dim": 128, "tokens": 2500, "past": 77, "max_seq": 4096},
        # the headline step's attention: one sequence, 129 keys
        {"name": "attend 1B 129 keys", "op": "attend", "rows": 1, "heads": 8, "group": 4, "dim": 64, "keys": 129, "max_seq": 256, "empty": False},
        # eight ragged sequences at the 1B shape's longest schedule
        {"name": "attend 1B 8x16384", "op": "attend", "rows": 8, "heads": 8, "group": 4, "dim": 64, "keys": 16384, "max_seq": 16384, "empty": False},
        # long texts with 128-wide heads, three queries a head, one row without keys
        {"name": "attend 128-wide 4x60001", "op": "attend", "rows": 4, "heads": 8, "group": 3, "dim": 128, "keys": 60001, "max_seq": 61440, "empty": True},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["select", "reorder", "append", "attend"])
    if op == "select":
        beams = rng.randint(1, 16)
        vocab = _spread(rng, 33, 131072)
        batch = max(1, min(_spread(rng, 1, 64), 12_000_000 // (beams * vocab)))
        n_out = min(rng.choice([1, beams, 2 * beams]), beams * vocab, 32)
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "n_out": n_out, "done": rng.randint(0, beams - 1)}
    dim = rng.choice([64, 128])
    heads = rng.choice([1, 2, 4, 8])
    if op == "reorder":
        bits = rng.choice([8, 16])
        seqs = rng.randint(1, 4)
        beams = rng.randint(2, 8 // seqs)
        layers = rng.randint(1, 28)
        per_slot = layers * heads * dim * seqs * beams * 2 * bits // 8
        length = _spread(rng, 200, max(201, min(16000, 900_000_000 // per_slot)))
        return {"op": op, "bits": bits, "layers": layers, "heads": heads, "dim": dim, "seqs": seqs, "beams": beams,
                "max_seq": length + rng.randint(1, 99), "length": length, "start": rng.choice([0, length // 3, length - 150])}
    if op == "append":
        layers, rows = rng.randint(1, 16), rng.randint(1, 8)
        tokens = _spread(rng, 1, max(2, min(8000, 120_000_000 // (layers * rows * heads * dim))))
        past = rng.choice([0, rng.randint(1, 31), rng.randint(1, 3000)])
        return {"op": op, "layers": layers, "rows": rows, "heads": heads, "dim": dim, "tokens": tokens, "past": past,
                "max_seq": past + tokens + 3 * T + rng.randint(0, 63)}
    rows = rng.randint(1, 8)
    keys = _spread(rng, 1, min(131072, 400_000_000 // (rows * heads * dim * 2)))
    return {"op": op, "rows": rows, "heads": heads, "group": rng.randint(1, 4), "dim": dim, "keys": keys,
            "max_seq": keys + rng.randint(0, 100), "empty": rows > 1 and rng.random() < 0.5}


# ------------------------------------------------------------------ what a case's data look like

def _row_lengths(case):
    """Valid slots of each row of a reorder case: the beams of one sequence are equally long."""
    return [max(1, case["length"] - 37 * (r // case["beams"])) for r in range(case["seqs"] * case["beams"])]


def _positions(case):
    """The last key of each row of an attend case: from all keys down to half of them, odd steps between."""
    n, rows = case["keys"], case["rows"]
    last = [n - 1 - (n * r) // (2 * rows) for r in range(rows)]
    if case["empty"]:
        last[rows // 2] = -1
    return last


def _counts(case):
    """New tokens of each row of an append case, ragged below the largest."""
    n = case["tokens"]
    return [n - (n * r) // (3 * case["rows"]) for r in range(case["rows"])]


def _firsts(case):
    """The first new slot of each row of an append case."""
    return [max(0, case["past"] - 13 * r) for r in range(case["rows"])]


def _parents(case, g):
    """The better half of each sequence's beams goes on twice, under any numbering of the beams."""
    beams, out = case["beams"], []
    for s in range(case["seqs"]):
        name = g.permutation(beams)
        to = np.empty(beams, dtype=np.int64)
        to[name] = name[np.arange(beams) // 2]
        out.extend(int(s * beams + p) for p in to)
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _codes(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen).mul_(42).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, gen):
    return torch.rand(shape, device="cuda", generator=gen).mul_(0.03).add_(0.015)


def _bf16(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16)


def _qcache(layers, rows, heads, max_seq, dim, gen):
    blocks = (max_seq + T - 1) // T
    return {"k_codes": _codes((layers, rows, heads, max_seq, dim), gen), "v_codes": _codes((layers, rows, heads, max_seq, dim), gen),
            "k_scale": _scales((layers, rows, heads, blocks), gen), "v_scale": _scales((layers, rows, heads, blocks), gen),
            "k_tail": _bf16((layers, rows, heads, T, dim), gen), "v_tail": _bf16((layers, rows, heads, T, dim), gen)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = np.random.default_rng(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "select":
        batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
        # a step's logits: a broad bulk, some tokens far above it
        x = torch.randn(batch * beams, vocab, device="cuda", generator=gen).mul_(2.0)
        peak = torch.randint(0, vocab, (batch * beams, 8), device="cuda", generator=gen)
        x.scatter_add_(1, peak, torch.rand(batch * beams, 8, device="cuda", generator=gen) * 12.0)
        s["logits"] = x
        s["scores"] = (torch.rand(batch, beams, device="cuda", generator=gen) * -20.0).contiguous()
        s["eos"] = vocab // 3
        done = np.zeros((batch, beams), dtype=np.int32)
        for row in done:
            row[g.permutation(beams)[:case["done"]]] = 1
        s["finished"] = _i32(done.tolist())
        n = case["n_out"]
        s["next_tokens"], s["parents"] = _i32([[0] * n] * batch), _i32([[0] * n] * batch)
        s["next_scores"] = torch.zeros(batch, n, device="cuda")
        s["next_finished"] = _i32([[0] * n] * batch)
        return s
    if op == "reorder":
        rows = case["seqs"] * case["beams"]
        shape = (case["layers"], rows, case["heads"], case["max_seq"], case["dim"])
        if case["bits"] == 16:
            s["k"], s["v"] = _bf16(shape, gen), _bf16(shape, gen)
        else:
            s.update(_qcache(*shape, gen))
        s["parents"] = _i32(_parents(case, g))
        s["lengths"], s["starts"] = _i32(_row_lengths(case)), _i32([case["start"]] * rows)
    elif op == "append":
        s.update(_qcache(case["layers"], case["rows"], case["heads"], case["max_seq"], case["dim"], gen))
        shape = (case["layers"], case["rows"], case["heads"], case["tokens"], case["dim"])
        s["k"], s["v"] = _bf16(shape, gen), _bf16(shape, gen)
        s["positions"], s["counts"] = _i32(_firsts(case)), _i32(_counts(case))
    else:
        s.update(_qcache(1, case["rows"], case["heads"], case["max_seq"], case["dim"], gen))
        n = case["heads"] * case["group"]
        s["q"] = torch.randn(case["rows"], n, case["dim"], device="cuda", generator=gen).mul_(2.0)
        s["positions"] = _i32(_positions(case))
        s["out"] = torch.zeros(case["rows"], n, case["dim"], device="cuda")
    if own and "k_codes" in s:
        from persistent_megakernel_interpreter_b200.qcache import QCache
        s["cache"] = QCache.from_tensors(*(s[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")))
        if op == "attend":
            s["workspace"] = s["cache"].attention_workspace(case["rows"], n, case["max_seq"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _RUN[s["op"]](s)


def _answer(s):
    if s["op"] == "reorder" and s["case"]["bits"] == 16:
        return [s["k"], s["v"]]
    return [s[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")]


def _run_select(s):
    if own:
        from persistent_megakernel_interpreter_b200.model import beam_select
        beam_select(s["logits"], s["scores"], s["next_tokens"], s["parents"], s["next_scores"], finished=s["finished"], eos=s["eos"],
                    next_finished=s["next_finished"])
        return [s["next_tokens"], s["parents"], s["next_scores"], s["next_finished"]]
    case, x, eos = s["case"], s["logits"], s["eos"]
    batch, beams, vocab, n = case["batch"], case["beams"], case["vocab"], case["n_out"]
    done = s["finished"].reshape(-1, 1) != 0
    # the rows' statistics, the sum and the totals in 64 bits: totals of different beams may lie close together
    top = x.amax(1, keepdim=True)
    total = torch.log(torch.exp(x - top).sum(1, keepdim=True, dtype=torch.float64))
    token = torch.arange(vocab, device="cuda")
    x = torch.where(done, torch.where(token == eos, 0.0, -math.inf), x)
    # the best of each row by logit, equal logits to the lower token: one whole number that orders both
    bits = x.view(torch.int32).to(torch.int64)
    bits = torch.where(x == 0, 0, torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits))
    row_n = min(n, vocab)
    key = torch.topk(bits * 2 ** 24 + (2 ** 24 - 1 - token), row_n, dim=1).values
    tok = 2 ** 24 - 1 - (key & (2 ** 24 - 1))
    logit = x.gather(1, tok).double()
    score = s["scores"].reshape(-1, 1).double()
    cand = torch.where(done, score + logit, score + ((logit - top.double()) - total)).reshape(batch, beams * row_n)
    # then of all rows, equal totals in the order of the rows
    best, at = torch.sort(cand, dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    parent = at // row_n + beams * torch.arange(batch, device="cuda")[:, None]
    tok = tok.reshape(batch, -1).gather(1, at)
    finished = (done.reshape(-1)[parent] | (tok == eos)).to(torch.int32)
    return [tok.to(torch.int32), parent.to(torch.int32), best.float(), finished]


def _reordered(t, parent, first, last):
    """t [layers][rows][heads][slots][...]: slots first .. last - 1 of each row from its parent, in place."""
    slot = torch.arange(t.shape[3], device="cuda")
    take = (slot >= first[:, None]) & (slot < last[:, None])
    take = take.reshape((1, take.shape[0], 1, take.shape[1]) + (1,) * (t.dim() - 4))
    t.copy_(torch.where(take, t.index_select(1, parent), t))


def _run_reorder(s):
    if own:
        if s["case"]["bits"] == 16:
            from persistent_megakernel_interpreter_b200.model import cache_reorder
            cache_reorder(s["k"], s["v"], s["parents"], s["lengths"], starts=s["starts"])
        else:
            s["cache"].reorder(s["parents"], s["lengths"], starts=s["starts"])
        return _answer(s)
    parent = s["parents"].long()
    last, first = s["lengths"].long()[parent], s["starts"].long()
    if s["case"]["bits"] == 16:
        _reordered(s["k"], parent, first, last)
        _reordered(s["v"], parent, first, last)
        return _answer(s)
    # closed blocks that hold any of the slots move whole, the open block's slots from its own first one
    closed, b0 = last // T, first // T
    for_open = torch.clamp(first - closed * T, min=0)
    _reordered(s["k_codes"], parent, b0 * T, closed * T)
    _reordered(s["v_codes"], parent, b0 * T, closed * T)
    _reordered(s["k_scale"], parent, b0, closed)
    _reordered(s["v_scale"], parent, b0, closed)
    _reordered(s["k_tail"], parent, for_open, last % T)
    _reordered(s["v_tail"], parent, for_open, last % T)
    return _answer(s)


def _append_one(codes, scales, tail, x, first, count):
    layers, rows, heads, max_seq, dim = codes.shape
    n = x.shape[3]
    blocks = (T - 1 + n + T - 1) // T
    held = first % T
    # a window from the start of each row's open block: its tokens so far, then the new ones
    at = torch.arange(blocks * T, device="cuda")
    from_new = torch.clamp(at - held[:, None], 0, n - 1)
    row = torch.arange(rows, device="cuda")[:, None]
    new = x[:, row, :, from_new].permute(2, 0, 3, 1, 4)  # [layers][rows][heads][window][dim]
    old = tail[:, :, :, torch.clamp(at, max=T - 1)]
    window = torch.where((at >= held[:, None])[None, :, None, :, None], new, old)
    part = window.float().reshape(layers, rows, heads, blocks, T * dim)
    big = part.abs().amax(4)
    some = big >= NO_BLOCK
    full = torch.full_like(big, 127.0)
    scale = torch.where(some, big / full, 0.0)
    code = torch.where(some[..., None], torch.round(part * (full / big)[..., None]), 0.0).clamp(-127, 127).to(torch.int8)
    # closed blocks into the cache; the others write back what is there
    block = torch.arange(blocks, device="cuda")
    close = ((block + 1) * T <= (held + count)[:, None])[None, :, None, :]
    to = first[:, None] // T + block
    layer, head = torch.arange(layers, device="cuda")[:, None, None, None], torch.arange(heads, device="cuda")[None, None, :, None]
    rw, to = row[None, :, None, :], to[None, :, None, :]
    scales[layer, rw, head, to] = torch.where(close, scale, scales[layer, rw, head, to])
    slot = to[..., None] * T + torch.arange(T, device="cuda")
    inside = torch.clamp(slot, max=max_seq - 1)
    code = code.reshape(layers, rows, heads, blocks, T, dim)
    where = (layer[..., None], rw[..., None], head[..., None], inside)
    codes[where] = torch.where(close[..., None, None], code, codes[where])
    # the tokens of the block that is open now
    end = held + count
    opened = end // T * T
    slot = torch.arange(T, device="cuda")
    fresh = (slot + opened[:, None] >= held[:, None]) & (slot + opened[:, None] < end[:, None])
    src = torch.clamp(slot + opened[:, None] - held[:, None], 0, n - 1)
    new = x[:, row, :, src].permute(2, 0, 3, 1, 4)
    tail.copy_(torch.where(fresh[None, :, None, :, None], new, tail))


def _run_append(s):
    if own:
        s["cache"].append(s["k"], s["v"], s["positions"], counts=s["counts"])
        return _answer(s)
    first, count = s["positions"].long(), s["counts"].long()
    _append_one(s["k_codes"], s["k_scale"], s["k_tail"], s["k"], first, count)
    _append_one(s["v_codes"], s["v_scale"], s["v_tail"], s["v"], first, count)
    return _answer(s)


def _run_attend(s):
    case = s["case"]
    if own:
        s["cache"].attention(0, s["q"], s["positions"], s["out"], max_ctx=case["max_seq"], workspace=s["workspace"])
        return s["out"]
    rows, heads, group, dim = case["rows"], case["heads"], case["group"], case["dim"]
    keys = (s["positions"].long() + 1)[:, None, None, None]
    last = case["keys"]
    slot = torch.arange(last, device="cuda")
    closed = (keys // T * T)[..., 0]
    is_open = (slot >= closed)[..., None]

    def whole(codes, scale, tail):  # the values that are held, in 32 bits
        x = codes[0, :, :, :last].float() * scale[0].repeat_interleave(T, 2)[:, :, :last, None]
        return torch.where(is_open, tail[0][:, :, slot % T].float(), x)

    q = s["q"].reshape(rows, heads, group, dim)
    score = (q @ whole(s["k_codes"], s["k_scale"], s["k_tail"]).transpose(2, 3)) / math.sqrt(dim)
    score = torch.where(slot < keys, score, -math.inf)
    top = torch.clamp(score.amax(3, keepdim=True), min=-1e30)  # a row without keys stays at weights of zero
    p = torch.exp(score - top)
    p = p / torch.clamp(p.sum(3, keepdim=True), min=1e-30)
    v = whole(s["v_codes"], s["v_scale"], s["v_tail"])
    return (p @ v).reshape(rows, heads * group, dim)


_RUN = {"select": _run_select, "reorder": _run_reorder, "append": _run_append, "attend": _run_attend}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "select":
        n = case["batch"] * (case["beams"] - case["done"]) * case["vocab"]
        return {"bytes": 4 * n + case["batch"] * (8 * case["beams"] + 16 * case["n_out"]), "flops": 4 * n}
    if op == "reorder":
        slots = 0
        lens = _row_lengths(case)
        for q in range(case["seqs"]):
            length = lens[q * case["beams"]]
            moved = case["beams"] - 1                      # every beam but the first changes
            sources = (case["beams"] - 1) // 2 + 1         # distinct parents of those
            slots += max(0, length - case["start"]) * (moved + sources)
        return {"bytes": slots * case["layers"] * case["heads"] * case["dim"] * 2 * case["bits"] // 8, "flops": 0}
    if op == "append":
        n = sum(_counts(case)) * case["layers"] * case["heads"]
        return {"bytes": 2 * n * (3 * case["dim"] + 4 / T), "flops": 2 * 3 * n * case["dim"]}
    keys = sum(p + 1 for p in _positions(case))
    heads = case["heads"] * case["group"]
    return {"bytes": 2 * keys * case["heads"] * case["dim"] + 2 * keys * case["heads"] * 4 / T + 8 * case["rows"] * heads * case["dim"],
            "flops": 4 * keys * heads * case["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_select(case, s):
    batch, beams, vocab, n = case["batch"], case["beams"], case["vocab"], case["n_out"]
    x, score = s["logits"].cpu().numpy(), s["scores"].cpu().numpy().astype(np.float64)
    done = s["finished"].cpu().numpy()
    out = np.empty((batch, n))
    for b in range(batch):
        pool = []
        for k in range(beams):
            if done[b, k]:
                pool.append(np.concatenate([[score[b, k]], np.full(min(n, vocab) - 1, -np.inf)]))
                continue
            row = x[b * beams + k].astype(np.float64)
            z = row.max() + np.log(np.sum(np.exp(row - row.max())))
            pool.append(score[b, k] + np.partition(row, vocab - min(n, vocab))[vocab - min(n, vocab):] - z)
        out[b] = np.sort(np.concatenate(pool))[::-1][:n]
    return [None, None, torch.from_numpy(out), None]


def _exact_reorder(case, s):
    parent, last, first = (s[n].tolist() for n in ("parents", "lengths", "starts"))
    if case["bits"] == 8:
        moved = []
        for name in ("k_scale", "v_scale", "k_tail", "v_tail"):
            old, new = s[name], s[name].double()
            for r, p in enumerate(parent):
                n = last[p] // T
                if name.endswith("scale"):
                    a, b = first[r] // T, n
                else:
                    a, b = max(0, first[r] - n * T), last[p] - n * T
                if a < b:
                    new[:, r, :, a:b] = old[:, p, :, a:b].double()
            moved.append(new)
        return [None, None, *moved]
    k, v = s["k"].clone(), s["v"].clone()
    for r, p in enumerate(parent):
        k[:, r, :, first[r]:last[p]] = s["k"][:, p, :, first[r]:last[p]]
        v[:, r, :, first[r]:last[p]] = s["v"][:, p, :, first[r]:last[p]]
    return [k.double(), v.double()] if k.numel() < 200_000_000 else [k, v]


def _exact_append(case, s):
    first, count = s["positions"].tolist(), s["counts"].tolist()
    scales, tails = [], []
    for name in ("k", "v"):
        scale, tail = s[name + "_scale"].double(), s[name + "_tail"].double()
        for r, (p, c) in enumerate(zip(first, count)):
            text = torch.cat([tail[:, r, :, :p % T], s[name][:, r, :, :c].double()], dim=2)
            n = text.shape[2] // T
            if n:
                big = text[:, :, :n * T].reshape(text.shape[0], text.shape[1], n, -1).abs().amax(3)
                scale[:, r, :, p // T:p // T + n] = torch.where(big < NO_BLOCK, 0.0, big / 127)
            rest = text.shape[2] - n * T
            tail[:, r, :, :rest] = text[:, :, n * T:]
        scales.append(scale)
        tails.append(tail)
    return [None, None, *scales, *tails]


def _exact_attend(case, s):
    rows, heads, group, dim = case["rows"], case["heads"], case["group"], case["dim"]
    out = torch.zeros(rows, heads, group, dim, dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(rows, heads, group, dim)
    for r, p in enumerate(s["positions"].tolist()):
        n = (p + 1) // T
        for h in range(heads if p >= 0 else 0):
            held = []
            for name in ("k", "v"):
                c = s[name + "_codes"][0, r, h, :n * T].double().reshape(n, T * dim) * s[name + "_scale"][0, r, h, :n, None].double()
                held.append(torch.cat([c.reshape(n * T, dim), s[name + "_tail"][0, r, h, :(p + 1) % T].double()]))
            w = torch.softmax(held[0] @ q[r, h].T / dim ** 0.5, 0)
            out[r, h] = w.T @ held[1]
    return out.reshape(rows, heads * group, dim)


_EXACT = {"select": _exact_select, "reorder": _exact_reorder, "append": _exact_append, "attend": _exact_attend}
