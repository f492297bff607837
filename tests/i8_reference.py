"""The 8-bit projection path's definition in numpy: integers decided in 64
bits, sums of integers exact, and the roundings to fp32 and bf16 that the
definition itself names."""
import numpy as np
import torch


def bf16(a):
    """fp32 values rounded to bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).float().numpy()


def rows(x, residual=None, weight=None, eps=1e-6, residual_bf16=False):
    """(q, scale in 64 bits, h) of fp32 rows x [M, D]."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        h = x if residual is None else x + np.asarray(residual, np.float32)
        if residual_bf16:
            h = bf16(h)
        a = h if weight is None else h * np.asarray(weight, np.float32)[None, :]
        bad = ~np.isfinite(a).all(1)
        m = np.abs(np.where(bad[:, None], 0, a)).max(1).astype(np.float64)
        # 127 a / m in 64 bits: a quotient of 24-bit numbers that is no half
        # is further than 2^-50 of it from one, so it rounds as the exact one
        t = 127.0 * np.where(bad[:, None], 0, a).astype(np.float64) / np.where(m > 0, m, 1)[:, None]
        q = np.rint(t).astype(np.int8)
        scale = m / 127.0
        if weight is not None:
            scale = scale / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1) + np.float64(np.float32(eps)))
        scale = np.where(bad, np.nan, np.where(m == 0, 0.0, scale))
    return q, scale, h


def linear(x, x_scale, w, w_scale, out_bf16=False):
    """fp32 values of the product, with the definition's roundings (bf16 too
    where asked). The sums are below 2^53, so the product in 64 bits is exact."""
    acc = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    with np.errstate(all="ignore"):
        y = acc.astype(np.float32) * np.asarray(x_scale, np.float32)[:, None]
        y = y * np.asarray(w_scale, np.float32)[None, :]
    return bf16(y) if out_bf16 else y
