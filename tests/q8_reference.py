"""8-bit caches and rotary positions in 64 bits on the CPU, from their definitions in pa.h."""
import numpy as np
import torch

from tests import attention_reference as ref

FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def e4m3_round(y):
    """Nearest e4m3 value (ties to even) of |y| <= 448: steps of 2^(e-3), e >= -6."""
    _, e = np.frexp(np.abs(y))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(y / step) * step


def quantise(fmt, x):
    """(codes as values, scales) of rows x [..., D]; the arithmetic is exact in float64 but for
    the int8 quotient, whose ties (127 x / t a half-integer) are exact too."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    x, top = np.where(bad, 0.0, x), np.where(bad, 0.0, top)
    if fmt == "e4m3":
        m, e = np.frexp(top / 448.0)  # exact: top <= 448 2^e
        e = np.maximum(np.where(m == 0.5, e - 1, e), -126)
        for d in (-1, 0, 1):  # top / 448 is rounded: take the least that holds
            fits = (top <= np.ldexp(448.0, e - 1)) & (e > -126)
            e = np.where(fits, e - 1, np.where(top > np.ldexp(448.0, e), e + 1, e))
        scale = np.ldexp(1.0, e)
        codes = e4m3_round(x / scale)
    else:
        t = np.maximum(top, 127.0 * 2.0 ** -126)
        scale = (t / 127.0).astype(np.float32).astype(np.float64)
        codes = np.round(127.0 * x / t)
    scale = np.where(top > 0, scale, 0.0)
    codes = np.where(top > 0, codes, 0.0)
    return codes, np.where(bad, np.nan, scale)[..., 0]


def rotate(x, positions, inv_freq, axes, adjacent, amplitude=1.0):
    """x [N, heads, D] float64, positions [axes, N]. Angles: the product of a 32-bit position and a
    float64 frequency is off by 2^-53 of itself, so whole turns are taken out of an exact
    integer product where positions are large (np.longdouble where it helps)."""
    y = np.array(x, np.float64)
    rot = 2 * len(inv_freq)
    ang = np.stack([positions[a].astype(np.longdouble) * np.longdouble(f)
                    for a, f in zip(axes, inv_freq)], -1)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    ang = (ang - np.round(ang / two_pi) * two_pi).astype(np.float64)
    c, s = amplitude * np.cos(ang)[:, None], amplitude * np.sin(ang)[:, None]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if adjacent else (y[..., :rot // 2],
                                                                y[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    if adjacent:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


def dequantised(codes, scales):
    """Rows [num_blocks * block_size, Hk, D] in float64."""
    x = codes.cpu().float().double() * scales.cpu().double().transpose(1, 2)[..., None]
    return x.reshape(-1, *x.shape[2:]).numpy()


def decode(q, k_rows, v_rows, v_scale_top, tables, lens, bs, out_dtype, scale=None, code_max=448.0,
           k_scale_top=0.0):
    """(out, tolerance) of pa_decode_q8. Beyond attention_reference's bound for the scores: each
    weight p vs is rounded to fp16, 2^-11 relative (with fp16 results to two fp16 numbers, 2^-22) or
    2^-39 of the largest value scale, times a code of at most code_max, once for each key; the
    output is rounded once to its type.

    int8 codes x enter the scores as 1152 + x, and the sums start at -1152 sum q: the D / 16 MMAs of
    a sum each round (or truncate) twice at most, 2^-23 of partial sums that reach
    (1152 + 1152 + 127) sum |q|, in units of scale times the key's scale."""
    q = q.double().cpu().numpy()
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    half = torch.finfo(out_dtype).eps / 2
    for b, n in enumerate(lens):
        t = np.arange(n)
        rows = np.asarray(tables[b])[t // bs].astype(np.int64) * bs + t % bs
        o, A, dev = ref.attend(q[b:b + 1], k_rows[rows], v_rows[rows], [n - 1],
                               np.ones((1, n), bool), scale=scale)
        out[b] = o[0]
        if code_max == 127.0:
            d = q.shape[-1]
            factor = d ** -0.5 if scale is None else scale
            dev = dev + (2 * (d // 16) * 2.0 ** -23 * 2431 * np.abs(q[b]).sum(-1)[None, :, None]
                         * factor * k_scale_top)
        weights = (2.0 ** -22 if out_dtype == torch.float16 else 2.0 ** -11) * A + n * code_max * 2.0 ** -39 * v_scale_top
        tol[b] = (half * np.abs(o) + (1 + half) * (weights + np.expm1(2 * dev) * A)
                  + 2.0 ** -25)[0]
    return out, tol
