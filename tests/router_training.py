"""The router's balance loss and the gradients of its logits from their
definitions in binary64 (NumPy), for the tests."""
import numpy as np


def sigmoid_parts(x):
    """(log sigmoid, 1 - sigmoid) of float64 logits; exact far into both tails."""
    with np.errstate(over="ignore"):
        u = np.exp(-np.abs(x))
        return np.minimum(x, 0) - np.log1p(u), np.where(x >= 0, u / (1 + u), 1 / (1 + u))


def relative_sigmoids(x):
    """(sigmoids of a row over the row's largest, 1 - sigmoids); a row of -inf is all zero."""
    ls, one_minus = sigmoid_parts(x)
    m = ls.max()
    return (np.zeros_like(x) if m == -np.inf else np.exp(ls - m)), one_minus


def offsets_of(offsets, T):
    return [0, T] if offsets is None else list(offsets)


def balance(logits, ids, mask, coeff, offsets=None):
    """-> (loss, counts [Q, E], prob_sums [Q, E], seq_tokens [Q])."""
    T, E = logits.shape
    k = ids.shape[1]
    cuts = offsets_of(offsets, T)
    Q = len(cuts) - 1
    counts, probs = np.zeros((Q, E), np.int64), np.zeros((Q, E))
    n = np.zeros(Q, np.int64)
    for q in range(Q):
        for t in range(cuts[q], cuts[q + 1]):
            if not mask[t]:
                continue
            n[q] += 1
            s, _ = relative_sigmoids(logits[t].astype(np.float64))
            if s.sum() > 0:
                probs[q] += s / s.sum()
            for i in ids[t]:
                if 0 <= i < E:
                    counts[q, i] += 1
    live = n > 0
    per = [E / (k * float(n[q]) ** 2) * float((counts[q] * probs[q]).sum()) for q in range(Q) if live[q]]
    return (coeff / len(per) * sum(per) if per else 0.0), counts, probs, n


def backward(logits, ids, mask, grad_w=None, grad_loss=None, coeff=0.0, counts=None, seq_tokens=None, offsets=None):
    """-> (gradient [T, E], magnitude [T, E]: the same sums over absolute terms)."""
    T, E = logits.shape
    k = ids.shape[1]
    grad, mag = np.zeros((T, E)), np.zeros((T, E))
    cuts = offsets_of(offsets, T)
    some = max(1, int((np.asarray(seq_tokens) > 0).sum())) if grad_loss is not None else 1
    for t in range(T):
        if not mask[t]:
            continue
        s, om = relative_sigmoids(logits[t].astype(np.float64))
        if grad_loss is not None:
            for q in range(len(cuts) - 1):
                if cuts[q] <= t < cuts[q + 1] and seq_tokens[q] > 0 and s.sum() > 0:
                    g = grad_loss * coeff / some * E / (k * float(seq_tokens[q]) ** 2) * counts[q]
                    G = (g * s).sum() / s.sum()
                    grad[t] += (g - G) * s * om / s.sum()
                    mag[t] += (g + abs(G)) * s * om / s.sum() if grad_loss >= 0 else (-g + abs(G)) * s * om / s.sum()
        if grad_w is not None:
            ok = [j for j in range(k) if 0 <= ids[t, j] < E]
            if ok:
                at = ids[t, ok]
                sj = np.exp(sigmoid_parts(logits[t, at].astype(np.float64))[0] -
                            sigmoid_parts(logits[t, at].astype(np.float64))[0].max()) \
                    if np.max(logits[t, at]) > -np.inf else np.zeros(len(at))
                w = sj / sj.sum() if sj.sum() > 0 else sj
                dw = grad_w[t, ok].astype(np.float64)
                np.add.at(grad[t], at, w * om[at] * (dw - (dw * w).sum()))
                np.add.at(mag[t], at, w * om[at] * (np.abs(dw) + (np.abs(dw) * w).sum()))
    return grad, mag
