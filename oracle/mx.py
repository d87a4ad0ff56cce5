"""Microscaled quantisation (oracle side, test infrastructure), from its formula in float64: per 32 columns the smallest
power of two 2^s with max|x| / 2^s <= the format's largest value, s in [-127, 127], and x / 2^s rounded to the format's
nearest value, ties to the even code; a block with a NaN or an infinity has scale code 255 and codes 0."""
from __future__ import annotations

import numpy as np

from .formats import E2M1_MAX, E2M1_TABLE, E4M3_MAX, bf16_rne, encode_e4m3_rne


def encode_e2m1_rne(v):
    """Codes of real values |v| <= 6: the nearest of the table's values, of two as near the even code."""
    a = np.abs(np.asarray(v, np.float64))
    d = np.abs(a[..., None] - E2M1_TABLE[:8])
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1)).astype(np.uint8)
    return np.where(np.signbit(v), code | 8, code).astype(np.uint8)


def mx_quant_ref(x, fmt):
    """(codes [R, C], one to a byte, scale codes [R, C / 32], the values they stand for as float32 rounded to BF16)."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    b = x.reshape(R, C // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top, most = np.abs(b).max(-1), {"e2m1": E2M1_MAX, "e4m3": E4M3_MAX}[fmt]
    s = np.full(top.shape, -127)
    for e in range(-126, 128):  # by trial, no logarithm: the first power that is enough
        s = np.where(top > most * np.ldexp(1.0, s), e, s)
    v = np.ldexp(b, -s[..., None])
    codes = encode_e2m1_rne(v) if fmt == "e2m1" else encode_e4m3_rne(v)
    table = E2M1_TABLE
    if fmt == "e4m3":
        from .formats import E4M3_TABLE as table
    with np.errstate(over="ignore"):
        dq = np.where(bad[..., None], np.nan, np.ldexp(table[codes], s[..., None]))
        dq = np.where(np.isnan(dq), np.nan, bf16_rne(dq.astype(np.float32)))
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(R, C), np.where(bad, 255, s + 127).astype(np.uint8), dq.reshape(R, C)
