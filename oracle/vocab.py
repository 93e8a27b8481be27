"""Losses over the vocabulary in float64, by their definitions (test
infrastructure only).  Logits z [M, V]; -inf is a masked word."""

import numpy as np


def log_softmax(z):
    """log p [M, V]; a row that is all -inf has log p = -inf."""
    z = np.asarray(z, np.float64)
    top = z.max(1, keepdims=True)
    dead = np.isneginf(top)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = z - np.where(dead, 0.0, top)
        lp = d - np.log(np.exp(d).sum(1, keepdims=True))
    return np.where(dead, -np.inf, lp)


def logprobs(z, target, top):
    """(logprob [M], entropy [M], top_logprob [M, top], top_index [M, top])."""
    z = np.asarray(z, np.float64)
    M, V = z.shape
    lp = log_softmax(z)
    real = (target >= 0) & (target < V)
    picked = np.where(real, lp[np.arange(M), np.where(real, target, 0)], 0.0)
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        h = -np.where(p > 0, p * lp, 0.0).sum(1)
    index = np.argsort(-z, axis=1, kind="stable")[:, :top]
    return picked, h, np.take_along_axis(lp, index, 1), index


def logprobs_grad(z, target, g_logprob, g_entropy):
    z = np.asarray(z, np.float64)
    M, V = z.shape
    lp = log_softmax(z)
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        plp = np.where(p > 0, p * lp, 0.0)
    h = -plp.sum(1, keepdims=True)
    alive = ~np.isneginf(z.max(1))
    real = (target >= 0) & (target < V) & alive
    gl = np.where(real, g_logprob, 0.0)[:, None]
    d = -p * gl - np.asarray(g_entropy, np.float64)[:, None] * (plp + p * h)
    d[np.arange(M)[real], target[real]] += gl[real, 0]
    return d


def distill(z, index, logit, temperature, weight):
    """(loss [M], gradient [M, V] of sum weight * loss)."""
    z = np.asarray(z, np.float64) / temperature
    M, V = z.shape
    t = np.asarray(logit, np.float64) / temperature
    real = (index >= 0) & (index < V)
    t = np.where(real, t, -np.inf)
    logq = log_softmax(t)
    q = np.exp(logq)
    lp = log_softmax(z)
    at = np.where(real, index, 0)
    with np.errstate(invalid="ignore"):
        loss = np.where(q > 0, q * (logq - np.take_along_axis(lp, at, 1)), 0.0).sum(1)
    d = np.exp(lp) * (q.sum(1, keepdims=True) > 0)
    for m in range(M):
        np.add.at(d[m], at[m], -q[m])
    d *= (np.asarray(weight, np.float64) / temperature)[:, None]
    d[np.isneginf(z.max(1))] = 0.0
    return loss, d
