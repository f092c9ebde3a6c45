"""Log probabilities of given tokens, entropy and top alternatives, oracle
side (test infrastructure only), in float64 from the definition: for a row of
logits x, ``p_i = exp(x_i) / sum exp(x)``; ``logprob = log p[token]``;
``entropy = -sum p log p`` with ``0 log 0 = 0``; the alternatives are the
largest logits, ties going to the lowest index (-0.0 equals +0.0)."""

import numpy as np


def row_logprobs(x):
    x = np.asarray(x, dtype=np.float64)
    m = x.max(axis=-1, keepdims=True)
    return (x - m) - np.log(np.exp(x - m).sum(axis=-1, keepdims=True))


def token_logprobs(x, tokens, top):
    """(logprob [N], entropy [N], top_ids [N, top], top_logprobs [N, top])."""
    lp = row_logprobs(x)
    n = lp.shape[0]
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(axis=-1)
    order = np.argsort(-(np.asarray(x, np.float64) + 0.0), axis=-1, kind="stable")[:, :top]
    return lp[np.arange(n), tokens], entropy, order, np.take_along_axis(lp, order, axis=-1)
