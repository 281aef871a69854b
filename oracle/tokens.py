"""Log probabilities of tokens in float64 (NumPy), with their gradient (test infrastructure).

Parity: pinned (gradients by differences; uniform and one-hot rows in closed form).
"""
import numpy as np


def forward(x, targets):
    """(logprob, entropy, maximum, log of the sum, log probabilities) of rows of logits."""
    x = np.asarray(x, dtype=np.float64)
    big = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = x - big
        log_s = np.log(np.exp(y).sum(axis=1, keepdims=True))
        logp = y - log_s
        p = np.exp(logp)
        entropy = -np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0).sum(axis=1)
    t = np.asarray(targets)
    lp = np.where(t >= 0, logp[np.arange(len(t)), np.maximum(t, 0)], 0.0)
    return lp, entropy, big[:, 0], log_s[:, 0], logp


def top(x, k):
    """The k largest of each row, equal ones by their number."""
    x = np.asarray(x, dtype=np.float64)
    return np.argsort(-x, axis=1, kind="stable")[:, :k]


def backward(x, targets, dlogprob, dentropy, dlse):
    """The gradient of sum(dlogprob logprob + dentropy entropy + dlse lse)."""
    _, entropy, _, _, logp = forward(x, targets)
    p = np.exp(logp)
    finite = np.where(p > 0, logp, 0.0)
    t = np.asarray(targets)
    dl = np.where(t >= 0, dlogprob, 0.0)[:, None]
    dx = p * (np.asarray(dlse)[:, None] - dl)
    dx -= np.asarray(dentropy)[:, None] * p * (finite + entropy[:, None])
    dx[np.arange(len(t)), np.maximum(t, 0)] += dl[:, 0]
    return dx
