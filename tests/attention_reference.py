"""Plain attention in 64 bits on the CPU, with the score rules of pa_decode_mod and
pa_prefill_mod, and the error bound that the kernels' arithmetic implies.

Bound per output element, eps = torch.finfo(type).eps (a rounding is off by eps / 2
relative), A = the probability-weighted mean of |v|:
- the output is rounded once: eps/2 * |ref|; each probability is rounded to the element type
  before the second product: eps/2 * A;
- a score is off by at most d (natural log units), which moves the output by at most
  (e^(2d) - 1) A. d: the fp32 dot product over D exact products, D * 2^-23 * sum |q k| scale
  (2^-23: a tensor core may truncate); the exponent's argument and the exp2, 2^-21 (|x| + 1);
  with a cap, the tanh and its scaling, 2^-19 cap in all.
- fp16 results below the normal range: 2^-25."""
import numpy as np
import torch


def gather(cache, table, total):
    """Rows of positions 0..total-1 as float64 [total, Hk, D]."""
    bs = cache.shape[1]
    t = np.arange(total)
    rows = torch.from_numpy(table[t // bs].astype(np.int64) * bs + t % bs)
    return cache.reshape(-1, *cache.shape[2:])[rows].double().numpy()


def visible(p, total, causal=True, window=0, sink=0, prefix=0):
    """[len(p), total] mask of the keys that queries at positions p see."""
    t = np.arange(total)[None, :]
    p = np.asarray(p)[:, None]
    see = (t < prefix) | (t <= p) if causal else np.ones((p.shape[0], total), bool)
    if window:
        see = see & ((t > p - window) | (t < sink) | (t < prefix))
    return see


def attend(q, k, v, pos, see, scale=None, softcap=0.0, slopes=None):
    """q [n, H, D], k, v [total, Hk, D] (float64), pos [n], see [n, total] -> (out, A, d)."""
    n, H, D = q.shape
    total, Hk, _ = k.shape
    G = H // Hk
    scale = D ** -0.5 if scale is None else scale
    out, A, dev = (np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros((n, H, 1)))
    if total == 0:
        return out, A, dev
    dist = np.abs(np.asarray(pos)[:, None] - np.arange(total)[None, :])
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        kk = np.where(np.isfinite(kk), kk, 0.0)  # hidden rows may hold anything
        vv = np.where(np.isfinite(vv), vv, 0.0)
        x = q[:, h] @ kk.T * scale
        mag = np.abs(q[:, h]) @ np.abs(kk).T * abs(scale)
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[h]) * dist
        mag = np.where(see, mag, 0).max(1, keepdims=True)
        top = np.where(see, np.abs(x), 0).max(1, keepdims=True)
        dev[:, h] = D * 2.0 ** -23 * mag + 2.0 ** -21 * (top + 1) + 2.0 ** -19 * softcap
        x = np.where(see, x, -np.inf)
        m = x.max(1, keepdims=True)
        e = np.where(see, np.exp(x - np.where(np.isfinite(m), m, 0.0)), 0.0)
        l = e.sum(1, keepdims=True)
        w = e / np.where(l > 0, l, 1.0)
        out[:, h] = w @ vv
        A[:, h] = w @ np.abs(vv)
    return out, A, dev


def bound(ref, A, dev, dtype, roundings=1):
    """The error bound above; `roundings` of the probabilities (1 for one pass)."""
    half = torch.finfo(dtype).eps / 2
    return (half * np.abs(ref) + roundings * half * A + np.expm1(2 * dev) * A * (1 + half)
            + 2.0 ** -25)


def assert_within(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: {np.argwhere(~np.isfinite(got))[:5].tolist()}"
    over = np.abs(got - ref) / tol
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over.max() <= 1.0, (f"{what}: {over.max():.2f} of the bound at {at}: got {got[at]} "
                               f"ref {ref[at]} tol {tol[at]}; {(over > 1).sum()} over")
