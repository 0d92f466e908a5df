"""Plain 64-bit forms of beam selection, cache reordering and the 8-bit cache, for the tests."""
import numpy as np

BLOCK = 32
NO_BLOCK = 2.0 ** -60


def select(logits, scores, n_out, finished=None, eos=-1):
    """logits [batch * beams][vocab] and scores [batch][beams] (fp32 arrays): tokens, parents, totals (64-bit),
    finished, each [batch][n_out]. Order: total, then lower beam, larger logit, lower token."""
    batch, beams = scores.shape
    vocab = logits.shape[1]
    tok, par, tot, fin = [], [], [], []
    for b in range(batch):
        cand = []
        for k in range(beams):
            x = logits[b * beams + k].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            score = np.float64(scores[b, k])
            done = finished is not None and finished[b, k] != 0
            if done:
                x = np.full(vocab, -np.inf)
                x[eos] = 0.0
                total = np.where(x == 0.0, score, -np.inf)
            else:
                m = x.max()
                with np.errstate(invalid="ignore", divide="ignore"):
                    d = np.where(x == m, 0.0, x - m)
                    d = np.where(x == -np.inf, -np.inf, d)
                    total = score + (d - np.log(np.sum(np.exp(d))))
                total = np.where(np.isnan(total) | (x == -np.inf), -np.inf, total)
            best = np.lexsort((np.arange(vocab), -x))[:n_out]
            cand += [(-total[v], k, -x[v], int(v), done) for v in best]
        cand = sorted(cand, key=lambda c: c[:4])[:n_out]
        tok.append([c[3] for c in cand])
        par.append([b * beams + c[1] for c in cand])
        tot.append([-c[0] for c in cand])
        fin.append([int(c[4] or (finished is not None and c[3] == eos)) for c in cand])
    return np.array(tok), np.array(par), np.array(tot), np.array(fin)


def reorder(t, parents, ranges):
    """t [layers][rows][heads][slots]...: row r's slots ranges(parent, r) = (lo, hi) from its parent, all at once."""
    new = t.copy()
    rows = t.shape[1]
    for r, p in enumerate(parents):
        if 0 <= p < len(parents) and p != r and p < rows:
            lo, hi = ranges(p, r)
            if lo < hi:
                new[:, r, :, lo:hi] = t[:, p, :, lo:hi]
    return new


def quantise(x):
    """One block (any shape, fp32 values): (codes, scale), as the cache holds it."""
    x = x.astype(np.float32)
    big = np.float32(np.max(np.abs(x))) if x.size else np.float32(0)
    if not np.all(np.isfinite(x)):
        return None, np.float32(np.nan)
    if big < NO_BLOCK:
        return np.zeros(x.shape, np.int8), np.float32(0)
    inv = np.float32(127) / big
    return np.rint(x * inv).astype(np.int8), big / np.float32(127)


def attend(q, k, v):
    """q [heads][dim], k and v [n][dim] of one KV head, in 64 bits."""
    if k.shape[0] == 0:
        return np.zeros(q.shape)
    s = q.astype(np.float64) @ k.astype(np.float64).T / np.sqrt(q.shape[1])
    w = np.exp(s - s.max(axis=1, keepdims=True))
    return (w / w.sum(axis=1, keepdims=True)) @ v.astype(np.float64)
