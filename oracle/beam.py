"""fp64 reference of beam search's selection: every candidate of a sequence, in
order.  Plain numpy from the definition; shares no code with the GPU path.  Test
infrastructure only."""
from __future__ import annotations

import numpy as np


def totals(logits, scores, finished=None, eos=None):
    """[batch, beams, vocab] totals; -inf for what is no candidate."""
    logits, scores = np.asarray(logits, np.float64), np.asarray(scores, np.float64)
    out = np.full(logits.shape, -np.inf)
    for b in range(logits.shape[0]):
        for k in range(logits.shape[1]):
            score, row = scores[b, k], logits[b, k]
            if not np.isfinite(score):
                continue
            if finished is not None and finished[b, k]:
                out[b, k, eos] = score
            elif not np.any(np.isnan(row)) and row.max() < np.inf and row.max() > -np.inf:
                top = row.max()
                # (row - top) first: logits may be the lowest value of their type
                out[b, k] = score + ((row - top) - np.log(np.sum(np.exp(row - top))))
    return out


def select(logits, scores, n_out, finished=None, eos=None):
    """(scores, parents, tokens, finished) in fp64 and integers; ties by the lower beam,
    the larger logit, the lower token."""
    t = totals(logits, scores, finished, eos)
    batch, _, vocab = t.shape
    flat = t.reshape(batch, -1)
    logit = np.where(flat == -np.inf, 0.0, np.asarray(logits, np.float64).reshape(batch, -1))
    if finished is not None:
        logit[np.repeat(np.asarray(finished) != 0, vocab, 1)] = 0.0
    beam = np.arange(flat.shape[1]) // vocab
    at = np.stack([np.lexsort((-logit[b], beam, -flat[b]))[:n_out] for b in range(batch)])  # stable: then the place
    parents, tokens = at // vocab, at % vocab
    done = tokens == (-1 if eos is None else eos)
    if finished is not None:
        done |= np.take_along_axis(np.asarray(finished) != 0, parents, 1)
    return np.take_along_axis(flat, at, 1), parents, tokens, done
