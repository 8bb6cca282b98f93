"""8-bit KV cache and LM-head log probabilities — TEST INFRASTRUCTURE ONLY.

The pages describe neither; the definitions are the library's own
(include/vgv.h). Arithmetic in fp64 on exact inputs.

* A code c of a block of positions and head stands for c * a / Q, Q = 127
  (int8) or 448 (e4m3: 4 significant bits, exponents down to 2^-6, then steps of
  2^-9); a = the block's largest magnitude. Codes are round(x * Q / a) to the
  nearest code, ties to even; a block that holds earlier positions takes the
  larger of its magnitude and the new rows', its earlier codes becoming
  round(c * a_old / a_new).
* Attention: softmax(scale q.k) v over the positions a row sees; nothing seen: 0.
* Log probabilities: z - logsumexp(z), entropy -sum p log p.

Codes are handled as their values, [B, n_kv, L, dim]; ``pack``/``unpack`` go
between those and the library's byte order.
"""
import numpy as np

from .bf16 import widen

Q_OF = {"int8": 127.0, "e4m3": 448.0}


def to_grid(x, fmt):
    """The code value nearest to x, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.rint(x)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(x / step) * step


def _byte_places(L, D, is_v):
    p, d = np.arange(L)[:, None], np.arange(D)[None, :]
    if is_v:
        return p // 16 * 16 * D + d // 4 * 64 + p % 16 // 4 * 16 + d % 4 * 4 + p % 4
    return p // 16 * 16 * D + d // 64 * 1024 + p % 16 * 64 + d % 64


_E4M3 = np.array([(-1.0 if b & 128 else 1.0) * (2.0 ** -9 * (b & 7) if b & 0x78 == 0 else
                                                2.0 ** ((b >> 3 & 15) - 7) * (1 + (b & 7) / 8)) for b in range(256)])


def pack(codes, fmt, is_v):
    """Code values [B, h, L, D] -> bytes [B, h, L, D] in the library's order."""
    B, h, L, D = codes.shape
    if fmt == "int8":
        raw = codes.astype(np.int8).view(np.uint8)
    else:
        order = np.argsort(_E4M3[:127])
        raw = order[np.searchsorted(_E4M3[:127][order], np.abs(codes))].astype(np.uint8) | (np.signbit(codes).astype(np.uint8) << 7)
    out = np.empty((B, h, L * D), np.uint8)
    out[:, :, _byte_places(L, D, is_v)] = raw
    return out.reshape(B, h, L, D)


def unpack(raw, fmt, is_v):
    B, h, L, D = raw.shape
    b = np.ascontiguousarray(raw).view(np.uint8).reshape(B, h, L * D)[:, :, _byte_places(L, D, is_v)]
    return b.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3[b]


def append(codes, amax, rows, pos, n_new, block, fmt):
    """codes [B, h, L, D] values and amax [B, h, L / block], changed in place;
    rows [B, rows, h, D] fp64 (finite or not)."""
    Q = Q_OF[fmt]
    for b in range(codes.shape[0]):
        p, n = int(pos[b]), int(n_new[b])
        for k in range(p // block, (p + n - 1) // block + 1 if n else 0):
            lo, hi = max(p, k * block), min(p + n, (k + 1) * block)
            x = rows[b, lo - p:hi - p].transpose(1, 0, 2)  # [h, hi - lo, D]
            top = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=(1, 2))
            was = amax[b, :, k] if lo > k * block else np.zeros_like(top)
            now = np.maximum(was, top)
            div = np.where(now > 0, now, 1.0)[:, None, None]
            with np.errstate(invalid="ignore"):
                y = np.clip(np.nan_to_num(x * Q / div, nan=0.0, posinf=Q, neginf=-Q), -Q, Q)
            old = codes[b, :, k * block:lo]
            turned = to_grid(old * was[:, None, None] / div, fmt)
            codes[b, :, k * block:lo] = np.where((now > was)[:, None, None], turned, old)
            codes[b, :, lo:hi] = to_grid(y, fmt)
            amax[b, :, k] = now


def values(codes, amax, block, fmt):
    return codes * np.repeat(amax, block, axis=2)[..., None] / Q_OF[fmt]


def attention(q, k, v, lens, scale, first=None, n_new=None):
    """q [B, rows, H, D] fp64; k, v values [B, h, L, D]. Returns (o [B, rows, H,
    D], sum_p p |v| of the same shape, the largest sum |q||k| scale of each row
    [B, rows, H])."""
    B, rows, H, D = q.shape
    h = k.shape[1]
    o, mag, size = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3])
    for b in range(B):
        for i in range(rows if n_new is None else int(n_new[b])):
            lo, hi = 0 if first is None else int(first[b]), int(lens[b]) + i + 1
            if lo >= hi:
                continue
            for j in range(H):
                kk, vv = k[b, j // (H // h), lo:hi], v[b, j // (H // h), lo:hi]
                s = kk @ q[b, i, j] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, i, j], mag[b, i, j] = p @ vv, p @ np.abs(vv)
                size[b, i, j] = (np.abs(kk) @ np.abs(q[b, i, j])).max() * scale
    return o, mag, size


def logprobs(h_bits, lm_bits):
    """(log p [R, V], entropy [R], sum_h |h W| [R, V]) in fp64."""
    h, w = widen(h_bits), widen(lm_bits)
    z = h @ w.T
    m = z.max(axis=1, keepdims=True)
    lp = z - (m + np.log(np.exp(z - m).sum(axis=1, keepdims=True)))
    return lp, -(np.exp(lp) * lp).sum(axis=1), np.abs(h) @ np.abs(w).T
