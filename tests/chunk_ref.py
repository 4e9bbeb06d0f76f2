"""Chunks of new tokens in 64 bits: the rotation, the append, and the attention over the cache, from their
definitions, with the bounds that the kernels' roundings give."""
import math

import torch

S = 128


def freqs(rope_dim, theta=10000.0, device="cuda"):
    return theta ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / max(1, rope_dim))


def rotate(x, pos, f, interleaved=False):
    """x [T][heads][d] in 64 bits, rotated to the positions; and the length of each element's pair."""
    R = 2 * len(f)
    y, size = x.double().clone(), x.double().abs()
    if R == 0:
        return y, size
    one, two = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a = pos.double().view(-1, 1, 1) * f
    u, v = x[..., one].double(), x[..., two].double()
    y[..., one], y[..., two] = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    size[..., one] = size[..., two] = torch.hypot(u, v)
    return y, size


def rotation_bound(y, size, dtype):
    """Half a step of the held value, and of fp32: sine and cosine to 2^-22, a product and a sum of two."""
    half = torch.finfo(dtype).eps / 2
    return half * y.abs() + 2.0 ** -21 * size * (1 + half)


class Case:
    """A paged cache in which every request holds past + n tokens, pages shuffled; behind each request's last
    token, and in pages that nobody maps, `fill`."""

    def __init__(self, reqs, Hq=8, Hkv=2, d=128, dtype=torch.bfloat16, seed=0, init=1024, local=7192,
                 fill=float("nan"), spare=3, slack=2, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.reqs, self.dtype = reqs, dtype
        self.cfg = dict(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=S, init_tokens=init,
                        local_tokens=local, topk_percent=0.2, dense_boundary=0,
                        dtype=int(dtype == torch.float32))
        blocks = [-(-(n + p) // S) for n, p in reqs]
        self.pages = sum(blocks) + spare
        perm = torch.randperm(self.pages, generator=g, device=device).int()
        self.max_blocks = max(1, max(blocks, default=1)) + slack
        self.table = torch.full((len(reqs), self.max_blocks), -7, dtype=torch.int32, device=device)
        at = 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = perm[at:at + b]
            at += b
        self.k, self.v = (torch.full((self.pages, Hkv, S, d), fill, device=device).to(dtype) for _ in "kv")
        for r, (n, p) in enumerate(reqs):
            for name in "kv":
                x = torch.randn(blocks[r] * S, Hkv, d, generator=g, device=device).to(dtype)
                x[n + p:] = fill
                getattr(self, name)[self.table[r, :blocks[r]].long()] = (
                    x.view(blocks[r], S, Hkv, d).transpose(1, 2).contiguous())
        ends = [0]
        for n, _ in reqs:
            ends.append(ends[-1] + n)
        self.T = ends[-1]
        self.offsets = torch.tensor(ends, dtype=torch.int32, device=device)
        self.past = torch.tensor([p for _, p in reqs], dtype=torch.int32, device=device)
        self.lens = torch.tensor([n + p for n, p in reqs], dtype=torch.int32, device=device)
        self.q = torch.randn(self.T, Hq, d, generator=g, device=device).to(dtype)
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)

    def tokens(self, r, length=None):
        """Request r's keys and values [length][Hkv][d] in 64 bits."""
        L = int(self.lens[r]) if length is None else length
        blocks = self.table[r, :-(-L // S)].long()
        return tuple(x[blocks].transpose(1, 2).flatten(0, 1)[:L].double() for x in (self.k, self.v))


def attention(case, window, rows=None):
    """out and the bound of its error, both [T][Hq][d] in 64 bits; rows outside every request are NaN."""
    c = case.cfg
    Hq, Hkv, d = c["num_q_heads"], c["num_kv_heads"], c["head_dim"]
    G = Hq // Hkv
    out = torch.full((case.T, Hq, d), float("nan"), dtype=torch.float64, device=case.q.device)
    tol = torch.zeros_like(out)
    half = torch.finfo(case.dtype).eps / 2
    for r in range(len(case.reqs)):
        lo, hi = int(case.offsets[r]), int(case.offsets[r + 1])
        n, L = hi - lo, int(case.lens[r])
        if n == 0:
            continue
        k, v = case.tokens(r)
        pos = torch.arange(L - n, L, device=out.device).unsqueeze(1)
        t = torch.arange(L, device=out.device)
        on = t <= pos
        if window:
            on &= (t < c["init_tokens"]) | (t > pos - c["local_tokens"])
        for j in range(Hq):
            q, kh, vh = case.q[lo:hi, j].double(), k[:, j // G], v[:, j // G]
            z = torch.where(on, q @ kh.T / math.sqrt(d), -math.inf)
            w = torch.where(on, torch.softmax(z, -1), 0.0)  # rows without a token: nothing
            # a token that no row attends may hold anything
            seen = on.any(0)
            vh = torch.where(seen.unsqueeze(1), vh, 0.0)
            o = w @ vh
            mass = w @ vh.abs()
            # logits: a sum of d products in fp32 (relative to the sum of their sizes), the scaling and the
            # exponential to some 2^-22; weights rounded once to the type; sums of L terms in fp32
            size = (q.abs() @ torch.where(seen.unsqueeze(1), kh, 0.0).abs().T / math.sqrt(d))
            size = torch.where(on, size, 0.0).amax(-1, keepdim=True) if L else 0.0
            delta = (d + 8) * 2.0 ** -24 * size + 2.0 ** -21
            p_half = half if case.dtype == torch.bfloat16 else 0.0
            out[lo:hi, j] = o
            tol[lo:hi, j] = half * o.abs() + mass * (1 + half) * (2 * p_half + 2 * delta + (L + 8) * 2.0 ** -24)
    return out, tol
