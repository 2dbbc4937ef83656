"""Oracle of beam search: the definition in float64 numpy, candidate by candidate."""
import numpy as np


def log_softmax(row):
    """Of one beam's logits in float64: NaN is masked, +inf has (its share of) everything."""
    row = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    top = row.max()
    if top == -np.inf:
        return row
    with np.errstate(invalid="ignore"):
        off = np.where(row == top, 0.0, row - top)
    return np.where(row == -np.inf, -np.inf, off - np.log(np.exp(off).sum()))


def select(logits, scores, count, finished=None, end=0):
    """[batch, beams, vocab] and [batch, beams]: scores (float64), parents and tokens, [batch, count]."""
    b, k, v = logits.shape
    out = np.zeros((b, count)), np.zeros((b, count), np.int32), np.zeros((b, count), np.int32)
    for i in range(b):
        S = np.full((k, v), -np.inf)
        for j in range(k):
            if finished is not None and finished[i, j]:
                S[j, end] = scores[i, j]
            else:
                with np.errstate(invalid="ignore"):
                    S[j] = np.float64(scores[i, j]) + log_softmax(logits[i, j])
        S = np.where(np.isnan(S), -np.inf, S)
        beam, token = np.divmod(np.arange(k * v), v)
        # of the last ones only their place counts
        logit = np.nan_to_num(np.where(S.ravel() == -np.inf, 0.0, logits[i].ravel().astype(np.float64)),
                              posinf=1e300)
        order = np.lexsort((token, -logit, beam, -S.ravel()))[:count]
        out[0][i], out[1][i], out[2][i] = S.ravel()[order], beam[order], token[order]
    return out


def reorder(state, parents):
    """state [batch, beams, ...]."""
    b, k = parents.shape
    p = np.where((parents >= 0) & (parents < k), parents, np.arange(k))
    return np.stack([state[i, p[i]] for i in range(b)]) if b else state
