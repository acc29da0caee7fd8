"""Float64 definitions of the paged cache's calls (rotary positions, 8-bit rows,
attention of one token) and of the sampling of a token.

Test infrastructure: numpy only, one sequence, head or row at a time."""
import numpy as np


def rotate(x, pos, freq):
    """Rows x [T, heads, D] with the first 2 len(freq) dimensions of a head turned by pos * freq."""
    x = np.array(x, dtype=np.float64)
    r = len(freq)
    a = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    u, w = x[..., :r].copy(), x[..., r:2 * r].copy()
    x[..., :r] = u * np.cos(a) - w * np.sin(a)
    x[..., r:2 * r] = w * np.cos(a) + u * np.sin(a)
    return x


def quantise(x):
    """8-bit rows along the last axis: codes and scales; a row with a NaN or an infinity: zeros and NaN."""
    m = np.abs(x).max(-1)
    fine = np.isfinite(m)
    safe = np.where(fine & (m > 0), m, 1.0)[..., None]
    q = np.where((fine & (m > 0))[..., None], np.rint(127.0 * np.where(fine[..., None], x, 0.0) / safe), 0.0)
    return q.astype(np.int8), np.where(fine, m / 127.0, np.nan)


def rows(pages, scales, table, page_rows, seq, pos):
    """Rows [T, heads, D] of the pages [n, heads, page_rows, D], in float64; zeros where there is no page."""
    out = np.zeros((len(pos), pages.shape[1], pages.shape[3]))
    for t, (s, p) in enumerate(zip(seq, pos)):
        page = table[s, p // page_rows] if 0 <= s < table.shape[0] and p // page_rows < table.shape[1] else -1
        if 0 <= page < pages.shape[0]:
            out[t] = pages[page, :, p % page_rows]
            if scales is not None:
                out[t] *= scales[page, :, p % page_rows, None].astype(np.float64)
    return out


def scores(q, k, scale, softcap=0.0):
    """Scores [L] of a query [D] and the sum of the products' magnitudes behind each."""
    z, size = scale * (k @ q), abs(scale) * (np.abs(k) @ np.abs(q))
    return (softcap * np.tanh(z / softcap) if softcap else z), size


def attend(q, k, v, scale, softcap=0.0):
    """One query [D] over keys and values [L, D]: the output, the log of the sum, the weighted mean of the
    values' magnitudes, and the largest sum of magnitudes behind a score."""
    if len(k) == 0:
        return np.zeros_like(q), -np.inf, np.zeros_like(q), 0.0
    z, size = scores(q, k, scale, softcap)
    p = np.exp(z - z.max())
    return p @ v / p.sum(), z.max() + np.log(p.sum()), p @ np.abs(v) / p.sum(), size.max()


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token and the log of its share of what remains; -1 and -inf where nothing does."""
    l = np.where(np.isfinite(logits), logits, -np.inf).astype(np.float64)  # (a +inf or NaN is left out)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if len(order) == 0:
        return -1, -np.inf
    if not temperature > 0:
        return int(order[0]), 0.0
    z = (l[order] - l[order[0]]) / float(temperature)
    if min_p > 0:
        z = z[z >= np.log(min(float(min_p), 1.0))]
    if top_k > 0:
        z = z[:top_k]
    w = np.exp(z)
    if top_p < 1:
        before = np.cumsum(w) - w
        w = w[(before < float(top_p) * w.sum()) | (np.arange(len(w)) == 0)]
    ids = np.argsort(order[:len(w)])
    at = np.cumsum(w[ids])
    pick = min(int(np.searchsorted(at, max(float(u), 0.0) * at[-1], side="right")), len(w) - 1)
    i = ids[pick]
    while w[i] == 0:  # past the end: the last one with a weight
        pick -= 1
        i = ids[pick]
    return int(order[i]), float(z[i] - np.log(w.sum()))
