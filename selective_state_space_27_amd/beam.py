"""Python binding of beam search on recurrent states (``include/mambascan.h``):
selection over beams and vocabulary, and the beams' states following their
parents.  Checks, streams and errors are as in norms.py; there is no autograd, and
it does not notice that reorder_states writes in place.
"""
from __future__ import annotations

import ctypes

import torch

import selective_state_space_27_amd as _mss

from .norms import _code, _on, _rows, _workspace_size
from .recurrence import _address, _marks, _state


def beam_select(logits, scores, n_out=None, *, finished=None, eos=None, stream=None):
    """The ``n_out`` (default: beams) best continuations of every sequence.

    total = scores + log_softmax(logits), over beams and vocabulary; in
    descending order, ties by the lower beam, then the larger logit (where 64 bits
    of a total do not tell them apart), then the lower token.  A beam's log sum
    is formed in fp32, so totals of two beams whose rows differ are told apart
    down to some 1e-7 (8.4e-6 each at most); below, their order is repeatable but
    not defined.  logits: [batch,
    beams, vocab] float32 or bfloat16 (rows may have a stride); scores: [batch,
    beams] float32, the beams' totals so far (-inf: not in use); finished:
    [batch, beams] bool or uint8, beams whose only candidate is the token
    ``eos`` at their score.  Banned tokens have logits of -inf; a beam with a NaN
    or +inf among its logits, or none above -inf, has no candidates.  Where a
    sequence has fewer candidates than n_out the rest have scores of -inf.

    Returns scores ([batch, n_out] float32), parents and tokens ([batch, n_out]
    int64), and with ``eos`` which of them are finished ([batch, n_out] bool)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3 or logits.numel() == 0:
        raise ValueError("logits must be a [batch, beams, vocab] tensor, none of them empty")
    dev = _mss._device_of(logits)
    batch, beams, vocab = logits.shape
    n = beams if n_out is None else n_out
    io = _code(logits.dtype)
    lp, ls = _rows(logits, "logits", logits.shape, logits.dtype, dev)
    if scores is None:
        raise TypeError("scores must be a torch.Tensor")
    sp = _state(scores, "scores", (batch, beams), dev)
    fp = _marks(finished, "finished", (batch, beams), dev)
    if eos is not None and not 0 <= eos < vocab:
        raise ValueError(f"eos {eos} is not in the vocabulary of {vocab}")
    if finished is not None and eos is None:
        raise ValueError("finished needs eos")
    need = _workspace_size("mss_beam_select_workspace_size", batch, beams, vocab, n)
    if need == 0:
        _mss._raise(5, "beam_select")
    handle, here = _on(stream, dev)
    with here:
        best = torch.empty((batch, n), dtype=torch.float32, device=dev)
        parents = torch.empty((batch, n), dtype=torch.int64, device=dev)
        tokens = torch.empty_like(parents)
        done = torch.empty((batch, n), dtype=torch.bool, device=dev) if eos is not None else None
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_beam_select(lp, ls, sp, fp, -1 if eos is None else eos,
                                        best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), _address(done), batch,
                                        beams, vocab, n, io, 0, ws.data_ptr(), need, handle)
    _mss._raise(st, "mss_beam_select")
    return (best, parents, tokens) if done is None else (best, parents, tokens, done)


def reorder_states(states, parents, *, stream=None):
    """states[s][b, k] = states[s][b, parents[b, k]], in place, for every tensor
    [batch, beams, ...] of ``states`` (contiguous, any type); parents: [batch,
    beams] int64.  Rows that stay where they are are not touched, nor are rows
    whose parent is outside 0 .. beams - 1.  Returns states."""
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2 or parents.numel() == 0:
        raise ValueError("parents must be a [batch, beams] tensor, neither of them empty")
    dev = _mss._device_of(parents)
    batch, beams = parents.shape
    _mss._check(parents, "parents", (batch, beams), torch.int64, dev)
    n = len(states)
    if n == 0:
        return states
    rows = []
    for i, t in enumerate(states):
        if not isinstance(t, torch.Tensor) or t.shape[:2] != parents.shape or t.numel() == 0:
            raise ValueError(f"states[{i}] must be a [batch, beams, ...] tensor with {batch} x {beams} rows, not empty")
        if t.device != dev or not t.is_contiguous():
            raise ValueError(f"states[{i}] must be contiguous and on {dev}")
        rows.append(t.numel() // (batch * beams) * t.element_size())
    handle, here = _on(stream, dev)
    with here:
        st = _mss.lib().mss_reorder_states((ctypes.c_void_p * n)(*(t.data_ptr() for t in states)),
                                           (ctypes.c_int64 * n)(*rows), n, parents.data_ptr(), batch, beams, handle)
    _mss._raise(st, "mss_reorder_states")
    return states
