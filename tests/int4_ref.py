"""The 4-bit page format and the decode over it in 64 bits (numpy), for the tests.

Written from the format's description in include/srkv.h, one code at a time: where word and bit of a
code lie comes from loops over tokens and elements, not from a layout trick."""
from __future__ import annotations

import numpy as np

S = 128


def bf16(a) -> np.ndarray:
    """bf16 bit patterns (uint16) as float64."""
    return (np.asarray(a, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def host(t) -> np.ndarray:
    """A bf16 torch tensor as float64."""
    import torch
    return bf16(t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16))


def to_bf16(x) -> np.ndarray:
    """float64 rounded once to bf16 (nearest, ties to even), as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        m, e = np.frexp(x)
        return np.where(np.isfinite(x), np.ldexp(np.rint(m * 256.0), e - 8), x)


def shift(j: int) -> int:
    return 4 * (j // 2) + 16 * (j % 2)


def slab_bytes(d: int) -> int:
    return 128 * d + 1024


def quantize_rows(x):
    """Rows x [..., d] (float64, bf16 values): codes [..., d] int64, scale and lo [...] float64."""
    x32 = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x32).all(-1)
        lo, hi = x32.min(-1), x32.max(-1)
        s = (hi - lo) / np.float32(15)
        up = ((s.view(np.uint32) + np.uint32(0xFFFF)) & np.uint32(0xFFFF0000)).view(np.float32)
        bad |= ~np.isfinite(np.float32(15) * up + np.abs(lo))
        diff = (x32 - lo[..., None]).astype(np.float64)
        q = diff / np.where(up > 0, up, 1).astype(np.float64)[..., None]
        codes = np.clip(np.rint(q), 0, 15)
    codes = np.where(bad[..., None] | (up == 0)[..., None], 0, codes).astype(np.int64)
    nan = np.float64("nan")
    return codes, np.where(bad, nan, up.astype(np.float64)), np.where(bad, nan, lo.astype(np.float64))


def unpack(slab: np.ndarray, d: int):
    """One slab (bytes): key codes, value codes [128][d], key scale, lo, value scale, lo [128]."""
    w = np.ascontiguousarray(slab).view(np.uint32)
    kw, vw = w[:16 * d].reshape(S, d // 8), w[16 * d:32 * d].reshape(4, d // 4, 4, 4)
    rows = np.ascontiguousarray(slab[S * d:]).view(np.uint16).reshape(2, S, 2)
    k, v = np.zeros((S, d), np.int64), np.zeros((S, d), np.int64)
    for j in range(8):
        k[:, j::8] = (kw >> np.uint32(shift(j))) & 15
    for t in range(S):
        words = vw[t // 32, :, (t % 32) // 8, :].reshape(d)
        v[t] = (words >> np.uint32(shift(t % 8))) & 15
    r = bf16(rows)
    return k, v, r[0, :, 0], r[0, :, 1], r[1, :, 0], r[1, :, 1]


def values(slab: np.ndarray, d: int):
    """One slab's keys and values [128][d] in float64."""
    k, v, ks, kl, vs, vl = unpack(slab, d)
    return kl[:, None] + k * ks[:, None], vl[:, None] + v * vs[:, None]


def decode_unit(q, kv, pages, L, sel, cfg, h):
    """One (request, kv head): outputs [G][d] in float64 and the error the kernel's arithmetic allows.

    q: [G][d] float64; kv: [P][Hkv][bytes]; pages: the request's block table row; sel: kept blocks.
    The bound, each rounding at half a step (finfo.eps / 2 of its type):
      * the output to bf16: 2^-8 |out|;
      * a weight times scale to fp16: 2^-11 of each, so 2^-11 of sum p vs c <= 2^-11 R with R the
        largest 15 vs; where it falls below fp16's normal range (scaled so that the largest is
        at least 4): half a subnormal step 2^-25 / 4 of the reference, N tokens of 15 codes: N 15 2^-27
        of the largest vs;
      * the query is exact in fp16 down to 2^-25 of its largest magnitude; below, 2^-25 of it each,
        at one part in 16 of the elements' scale: 2^-21 d |q|max 15 ks in a logit;
      * fp32 sums of d products and the parameters' products: (d + 8) 2^-23 of sum |q| (|klo| + 15 ks) in
        a logit (2^-23: the tensor cores' sums may truncate), and 2^-22 |z| in the exponential;
        a logit's error e moves the output by at most 2 e times the spread of the values;
      * fp32 sums over the tokens: (N / 8 + 64) 2^-23 of sum p (15 vs + |vlo|), numerator and sum.
    """
    d, G = q.shape[1], q.shape[0]
    INIT, LOCAL = cfg["init_tokens"], cfg["local_tokens"]
    W = L - LOCAL
    keep = set(int(b) for b in sel)
    K, V, par = [], [], []
    for b in range(-(-L // S)):
        t = np.arange(b * S, min(L, b * S + S))
        on = (t < INIT) | (t >= W) | ((b in keep) & (t >= INIT) & (t < W))
        if not on.any():
            continue
        k, v, ks, kl, vs, vl = unpack(kv[pages[b], h], d)
        n = len(t)
        K.append((kl[:n, None] + k[:n] * ks[:n, None])[on])
        V.append((vl[:n, None] + v[:n] * vs[:n, None])[on])
        par.append(np.stack([15 * ks[:n] + np.abs(kl[:n]), 15 * vs[:n], np.abs(vl[:n])], 1)[on])
    if not K:
        return np.zeros((G, d)), np.zeros((G, d))
    K, V, par = np.concatenate(K), np.concatenate(V), np.concatenate(par)
    z = q @ K.T / np.sqrt(d)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = p @ V
    N, qa = len(K), np.abs(q)
    R, lo, kmax = par[:, 1].max(), par[:, 2].max(), par[:, 0].max()
    dz = ((2.0 ** -21 * d * qa.max() + (d + 8) * 2.0 ** -23 * qa.sum(1)) * kmax / np.sqrt(d)
          + 2.0 ** -22 * np.abs(z).max(1))
    bound = (2.0 ** -8 * np.abs(out) + 2.0 ** -11 * R + N * 2.0 ** -27 * R
             + 2 * dz[:, None] * (R + 2 * lo) + 2 * (N / 8 + 64) * 2.0 ** -23 * (R + lo))
    return out, bound
