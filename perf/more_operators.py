"""What is measured of a prompt's way into the paged cache: a ragged chunk of new tokens rotated to its
positions and appended, and its attention over the cache, in full and with a sliding window and first tokens.

Request r of a batch brings the rows [offsets[r], offsets[r + 1]) of the packed inputs.  Appended at a length of
P tokens, row i stands at position p = P + i; attended, the length counts the new tokens, p = L - n + i.

    rotation  (x, y) -> (x cos a - y sin a, y cos a + x sin a),  a = p * freq[j], for the pairs (j, j + R / 2) of the
              first R elements, or (2j, 2j + 1) where interleaved; elements from R on stay as they are
    append    q' = rot(q), key row = rot(k), value row = v, each rounded once; a written page's vector = the mean of
              its keys as held, up to the last one written
    chunk     out = softmax over t <= p of q . k_t / sqrt(d), times v_t
    window    the same over those t <= p with t < init or t > p - local

The plain forms are elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

S = 128  # tokens a page
DEV = "cuda"
LOGITS = 1 << 29  # logits that a plain form holds at a time


# ---- cases --------------------------------------------------------------------------------------------

def listed():
    layer = dict(q_heads=32, heads=8, d=128, dtype="bf16", lead=0)
    small = dict(q_heads=15, heads=5, d=64, dtype="bf16", lead=0)
    return [
        # one request's new token in a decode loop, rotated and written in the middle of its page
        dict(layer, name="append 1", kind="append", batch=1, new_lo=1, new_hi=1, past_lo=65499, past_hi=65499, rope=128,
             inter=False),
        # a serving batch's new tokens, every request at another row of its page
        dict(layer, name="append 64 tokens", kind="append", batch=64, new_lo=1, new_hi=1, past_lo=2048, past_hi=8192,
             rope=128, inter=False),
        # the last chunk of a 65536-token prompt
        dict(layer, name="append 8192", kind="append", batch=1, new_lo=8192, new_hi=8192, past_lo=57344,
             past_hi=57344, rope=128, inter=False),
        # chunks of all lengths, empty ones among them, half of each head rotated in neighbouring pairs
        dict(small, name="append 13 ragged d64", kind="append", batch=13, new_lo=0, new_hi=700, past_lo=5001,
             past_hi=0, rope=32, inter=True),
        # a single token over everything before it: the 65536-token layer, no block left out
        dict(layer, name="chunk 1 of 65536", kind="chunk", batch=1, new_lo=1, new_hi=1, past_lo=65535, past_hi=65535),
        # a whole prompt in one chunk
        dict(layer, name="chunk prompt 4096", kind="chunk", batch=1, new_lo=4096, new_hi=4096, past_lo=0, past_hi=0),
        # the last chunk of a 131072-token prompt: the largest
        dict(layer, name="chunk 8192 of 131072", kind="chunk", batch=1, new_lo=8192, new_hi=8192, past_lo=122880,
             past_hi=122880),
        # a step of a serving batch: one request's prompt goes on by 2048 tokens, the others decode; groups of 8
        dict(layer, name="chunk 2048 and 31 tokens", kind="chunk", q_heads=64, batch=32, new_lo=1, new_hi=1,
             past_lo=16384, past_hi=2048, lead=2048),
        # odd chunks in full precision, an empty one among them
        dict(small, name="chunk 7 ragged d64 fp32", kind="chunk", dtype="fp32", batch=7, new_lo=0, new_hi=300,
             past_lo=4096, past_hi=0),
        # a decode batch that sees its window and the first tokens only
        dict(layer, name="window 64 tokens", kind="window", batch=64, new_lo=1, new_hi=1, past_lo=4000,
             past_hi=32768, init=1024, local=7192),
        # the last chunk of a 131072-token prompt, windowed
        dict(layer, name="window 8192 of 131072", kind="window", batch=1, new_lo=8192, new_hi=8192, past_lo=122880,
             past_hi=122880, init=1024, local=7192),
        # chunks of all lengths at odd bounds
        dict(small, name="window 13 ragged d64", kind="window", batch=13, new_lo=0, new_hi=700, past_lo=20000,
             past_hi=0, init=300, local=1111),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("append", "chunk", "chunk", "window", "window"))
    heads = rng.choice((1, 2, 3, 4, 5, 7, 8))
    case = dict(kind=kind, d=rng.choice((64, 128)), heads=heads, q_heads=heads * rng.choice((1, 2, 3, 4, 5, 8)),
                dtype=rng.choice(("bf16", "bf16", "bf16", "fp32")), batch=_log(rng, 1, 64), lead=0)
    wide = 4 if case["dtype"] == "fp32" else 1  # full precision: a sixteenth of the work
    new = _log(rng, 1, max(1, 8192 // wide // case["batch"]))
    ends = rng.choice(((new, new), (0, new), (new, 1))) if case["batch"] > 1 else (new, new)
    case["new_lo"], case["new_hi"] = ends
    past = _log(rng, 128, max(129, 131072 // wide // max(1, case["batch"] // 4)))
    case["past_lo"], case["past_hi"] = rng.choice(((past, past), (0, past), (past, past // 2), (past, 0)))
    if case["batch"] > 1 and rng.random() < 0.3:
        case["lead"] = _log(rng, 2, 4096 // wide)
    if kind == "append":
        case["rope"] = rng.choice((case["d"], case["d"], case["d"] // 2, 16))
        case["inter"] = rng.random() < 0.3
    if kind == "window":
        case["init"], case["local"] = rng.choice((0, 4, 64, 300, 1024)), rng.choice((1, 128, 500, 1111, 4096, 7192))
    if kind != "append":
        at_most = work(listed()[6])["flops"]
        while work(case)["flops"] > at_most / wide ** 2:
            case["past_lo"], case["past_hi"] = case["past_lo"] // 2, case["past_hi"] // 2
    return case


def _even(lo, hi, n):
    return [lo] * n if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _requests(case):
    """[(new tokens, tokens before them)], a leading request's longer chunk first."""
    new = _even(case["new_lo"], case["new_hi"], case["batch"])
    past = _even(case["past_lo"], case["past_hi"], case["batch"])
    if case["lead"]:
        new[0] = case["lead"]
    return list(zip(new, past))


def _bounds(case):
    """(first tokens, window) that every row sees; without a window the first tokens are all there are."""
    return (case["init"], case["local"]) if case["kind"] == "window" else (1 << 30, 0)


def work(case):
    d, H, Hq = case["d"], case["heads"], case["q_heads"]
    e = 4 if case["dtype"] == "fp32" else 2
    moved = flops = 0
    for n, past in _requests(case):
        if not n:
            continue
        if case["kind"] == "append":  # queries, keys and values in and out, the keys of the first page, the vectors
            pages = (past + n - 1) // S - past // S + 1
            moved += n * (2 * Hq + 4 * H) * d * e + past % S * H * d * e + pages * H * d * 4
            flops += n * (Hq + H) * case["rope"] * 3 + (n + past % S) * H * d
            continue
        init, local = _bounds(case)
        L, seen = past + n, init + local
        whole = min(n, max(0, seen - past))  # rows that see all before them
        flops += 4 * d * Hq * (whole * past + whole * (whole + 1) // 2 + (n - whole) * seen)
        tokens = min(L, init) + max(0, L - max(min(L, init), past + 1 - local))
        moved += (2 * n * Hq + 2 * tokens * H) * d * e
    return dict(bytes=moved, flops=flops)


# ---- inputs ---------------------------------------------------------------------------------------------

def _type(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _config(case):
    return dict(num_q_heads=case["q_heads"], num_kv_heads=case["heads"], head_dim=case["d"], block_size=S,
                init_tokens=case.get("init", 1024), local_tokens=case.get("local", 7192), topk_percent=0.2,
                dense_boundary=32768, dtype=int(case["dtype"] == "fp32"))


def _pages(g, pages, case):
    """Keys with a gain and an offset for each channel, as projections with a rotation leave them, and values."""
    H, d, dt = case["heads"], case["d"], _type(case)
    gain = torch.rand(H, 1, d, generator=g, device=DEV) + 0.5
    shift = torch.randn(H, 1, d, generator=g, device=DEV) * 0.5
    k, v = (torch.empty(pages, H, S, d, dtype=dt, device=DEV) for _ in "kv")
    for p in range(0, pages, 256):
        n = min(256, pages - p)
        k[p:p + n] = (torch.randn(n, H, S, d, generator=g, device=DEV) * gain + shift).to(dt)
        v[p:p + n] = torch.randn(n, H, S, d, generator=g, device=DEV).to(dt)
    return k, v


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    H, Hq, d, dt = case["heads"], case["q_heads"], case["d"], _type(case)
    reqs = _requests(case)
    st = dict(case=case, cfg=_config(case), reqs=reqs)
    ends = [0]
    for n, _ in reqs:
        ends.append(ends[-1] + n)
    T = ends[-1]
    st["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
    blocks = [-(-(n + past) // S) for n, past in reqs]
    # an append's table names only the pages that it touches: no others are in the cache
    first = [past // S if case["kind"] == "append" else 0 for _, past in reqs]
    held = [max(0, b - f) for b, f in zip(blocks, first)]
    pages = max(1, sum(held))
    perm, at = torch.randperm(pages, generator=g, device=DEV).int().cpu(), 0
    table = torch.full((len(reqs), max(1, max(blocks))), -1, dtype=torch.int32)
    for r, (f, n) in enumerate(zip(first, held)):
        table[r, f:f + n] = perm[at:at + n]
        at += n
    st["table"] = table.to(DEV)
    st["k"], st["v"] = _pages(g, pages, case)
    if case["kind"] == "append":
        st["lens"] = torch.tensor([past for _, past in reqs], dtype=torch.int32, device=DEV)
        # queries, keys and values side by side, as one projection leaves them
        qkv = torch.randn(T, Hq + 2 * H, d, generator=g, device=DEV).to(dt)
        st["q_new"], st["k_new"], st["v_new"] = qkv.split((Hq, H, H), 1)
        R = case["rope"]
        st["freqs"] = 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
        st["at"] = torch.tensor([past + i for n, past in reqs for i in range(n)], dtype=torch.float64, device=DEV)
        if dt == torch.bfloat16:
            _part_the_borders(st)
        st["reps"] = torch.zeros(pages, H, d, device=DEV)
        st["q_out"] = torch.zeros(T, Hq, d, dtype=dt, device=DEV)
        return st
    st["lens"] = torch.tensor([n + past for n, past in reqs], dtype=torch.int32, device=DEV)
    st["q"] = (torch.randn(T, Hq, d, generator=g, device=DEV) * 2).to(dt)
    st["out"] = torch.zeros(T, Hq, d, dtype=dt, device=DEV)
    if own:
        from block_sparse_retrieval_gb300 import srkv
        st["workspace"] = torch.empty(srkv.chunk_workspace_size(st["cfg"], T, len(reqs)), dtype=torch.uint8, device=DEV)
    return st


def _part_the_borders(st):
    """Moves a key's pair to the next values where its rotation lands within 2^-17 of a border between two bf16
    values: which of them is held, and with it the page's mean, then does not hang on a 32-bit product's last bits."""
    c, k = st["case"], st["k_new"]
    a = st["at"].view(-1, 1, 1) * st["freqs"]
    for turn in range(16):
        y, size = _turned_exactly(k, a, c["inter"])
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1e-30))) - 7)
        near = ((y / step - torch.floor(y / step) - 0.5).abs() * step < size * 2.0 ** -17)
        if not near.any():
            return
        one, two = _halves(c["rope"], c["inter"])
        near[..., one] |= near[..., two]  # both of the pair: the smaller one alone may not move it
        near[..., two] = near[..., one]
        x = k[..., :c["rope"]]
        x.copy_(torch.where(near, (x.view(torch.int16) ^ (1 + turn % 6)).view(torch.bfloat16), x))


def _halves(R, inter):
    return (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))


def _turned_exactly(x, a, inter):
    """The first elements of x in 64 bits, rotated by the angles a, and the lengths of the pairs."""
    R = 2 * a.shape[-1]
    one, two = _halves(R, inter)
    z = torch.complex(x[..., one].double(), x[..., two].double())
    z = z * torch.polar(torch.ones_like(a), a)
    y = torch.empty(*x.shape[:-1], R, dtype=torch.float64, device=x.device)
    size = torch.empty_like(y)
    y[..., one], y[..., two] = z.real, z.imag
    size[..., one] = size[..., two] = z.abs()
    return y, size


# ---- one pass -------------------------------------------------------------------------------------------

def run(st):
    kind = st["case"]["kind"]
    if own:
        from block_sparse_retrieval_gb300 import srkv
        if kind == "append":
            srkv.append_kv_rope(st["cfg"], st["q_new"], st["k_new"], st["v_new"], st["freqs"], st["k"], st["v"],
                                st["table"], st["offsets"], st["lens"], st["reps"], st["q_out"],
                                interleaved=st["case"]["inter"])
            return dict(q=st["q_out"], k=st["k"], v=st["v"], reps=st["reps"])
        call = srkv.chunk_attention if kind == "chunk" else srkv.chunk_attention_window
        call(st["cfg"], st["q"], st["k"], st["v"], st["table"], st["offsets"], st["lens"], st["out"], st["workspace"])
        return dict(out=st["out"])
    return _plain_append(st) if kind == "append" else _plain_attention(st)


def _plain_append(st):
    c, dt = st["case"], st["k"].dtype
    a = st["at"].view(-1, 1, 1) * st["freqs"]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    R = c["rope"]

    def turn(x):
        x = x.float()
        if c["inter"]:
            one, two = x[..., 0:R:2], x[..., 1:R:2]
            y = torch.stack((one * cos - two * sin, two * cos + one * sin), -1).flatten(-2)
        else:
            one, two = x[..., :R // 2], x[..., R // 2:R]
            y = torch.cat((one * cos - two * sin, two * cos + one * sin), -1)
        return torch.cat((y, x[..., R:]), -1).to(dt)

    st["q_out"].copy_(turn(st["q_new"]))
    n = st["offsets"].diff().long()
    r = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=len(st["at"]))
    pos = st["at"].long()
    page = st["table"][r, pos // S].long()
    st["k"][page, :, pos % S] = turn(st["k_new"])
    st["v"][page, :, pos % S] = st["v_new"]
    # the pages written, each once, with the keys that they hold now
    held = torch.zeros(len(st["k"]), dtype=torch.long, device=DEV).scatter_reduce_(0, page, pos % S + 1, "amax")
    on = torch.arange(S, device=DEV) < held.unsqueeze(1)
    mean = torch.where(on[:, None, :, None], st["k"].float(), 0).sum(2) / held.clamp(min=1).view(-1, 1, 1)
    st["reps"].copy_(torch.where((held > 0).view(-1, 1, 1), mean, st["reps"]))
    return dict(q=st["q_out"], k=st["k"], v=st["v"], reps=st["reps"])


def _slices(st, lanes):
    """(request, first row, rows, position of the first row, tokens from, tokens before which all are read) of
    pieces with at most LOGITS logits: a piece reads the first tokens below `init` and those from `from` on."""
    init, local = _bounds(st["case"])
    at = 0
    for r, (n, past) in enumerate(st["reqs"]):
        i = 0
        while i < n:
            rows = max(1, min(n - i, 1024 if local else n, LOGITS // (lanes * (past + n))))
            start = max(0, min(past + i + 1 - local, past + i + rows)) if local else 0
            yield r, at + i, rows, past + i, start, min(init, past + i + rows)
            i += rows
        at += n


def _tokens(st, r, start, first, end):
    """The tokens that a piece reads: [0, first) and [start, end)."""
    t = torch.arange(end, device=DEV)
    return t if start <= first else torch.cat((t[:first], t[start:]))


def _plain_attention(st):
    H, Hq, d = st["case"]["heads"], st["case"]["q_heads"], st["case"]["d"]
    init, local = _bounds(st["case"])
    for r, row, rows, p, start, first in _slices(st, Hq):
        t = _tokens(st, r, start, first, p + rows)
        page, at = st["table"][r, t // S].long(), t % S
        keys, vals = st["k"][page, :, at].float(), st["v"][page, :, at].float()  # [tokens][H][d]
        q = st["q"][row:row + rows].float().reshape(rows, H, Hq // H, d).permute(1, 2, 0, 3).reshape(H, -1, d)
        z = torch.matmul(q, keys.permute(1, 2, 0)) / math.sqrt(d)
        pos = torch.arange(p, p + rows, device=DEV).unsqueeze(1)
        on = (t <= pos) & ((t < init) | (t > pos - local))
        z = torch.where(on, z.view(H, Hq // H, rows, -1), -math.inf)
        top = z.amax(-1, keepdim=True)
        w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.view(H, -1, w.shape[-1]), vals.transpose(0, 1)).view(H, Hq // H, rows, d)
        o = o / torch.where(total > 0, total, 1.0)
        st["out"][row:row + rows] = o.permute(2, 0, 1, 3).reshape(rows, Hq, d).to(st["out"].dtype)
    return dict(out=st["out"])


# ---- in 64 bits -----------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    H, Hq, d = case["heads"], case["q_heads"], case["d"]
    G = Hq // H
    if case["kind"] == "append":
        a = st["at"].view(-1, 1, 1) * st["freqs"]
        R = case["rope"]
        q, k, v = st["q_new"].double(), st["k_new"].double(), st["v"].double()
        q[..., :R], k[..., :R] = _turned_exactly(q, a, case["inter"])[0], _turned_exactly(k, a, case["inter"])[0]
        keys, held, reps = st["k"].double(), st["k"].double(), st["reps"].double()
        row = 0
        for r, (n, past) in enumerate(st["reqs"]):
            for b in range(past // S, -(-(past + n) // S) if n else 0):
                lo, hi = max(past, b * S), min(past + n, b * S + S)
                page, new = int(st["table"][r, b]), slice(row + lo - past, row + hi - past)
                keys[page, :, lo - b * S:hi - b * S] = k[new].transpose(0, 1)
                held[page, :, lo - b * S:hi - b * S] = k[new].to(st["k"].dtype).double().transpose(0, 1)
                v[page, :, lo - b * S:hi - b * S] = st["v_new"][new].double().transpose(0, 1)
                reps[page] = held[page, :, :hi - b * S].mean(1)
            row += n
        return dict(q=q, k=keys, v=v, reps=reps)
    init, local = _bounds(case)
    pieces = []  # (request, first row of the chunk, rows, its position); of a window's rows, few at a time
    row = 0
    for r, (n, past) in enumerate(st["reqs"]):
        step = 512 if local else 2048
        pieces += [(r, row + i, min(step, n - i), past + i) for i in range(0, n, step)]
        row += n
    if sum(4.0 * m * min(p + m, 2 * init + local + m) * Hq * d for _, _, m, p in pieces) > 6e12:
        return None
    out = torch.zeros(row, Hq, d, dtype=torch.float64, device=DEV)
    for r, at, m, p in pieces:
        seen = torch.arange(p + m, device=DEV)
        if local:
            seen = seen[(seen < init) | (seen > p - local)]
        slot, place = torch.div(seen, S, rounding_mode="floor"), torch.remainder(seen, S)
        slot = st["table"][r].long()[slot]
        i = torch.arange(p, p + m, device=DEV)
        hidden = (seen[None] > i[:, None]) | ((seen[None] >= init) & (seen[None] <= i[:, None] - local))
        for h in range(H):
            kh, vh = st["k"][slot, h, place].double(), st["v"][slot, h, place].double()
            for j in range(h * G, h * G + G):
                z = (st["q"][at:at + m, j].double() @ kh.T * d ** -0.5).masked_fill_(hidden, -math.inf)
                w = torch.softmax(z, -1).nan_to_num_(0.0)  # a row that sees nothing gives zeros
                out[at:at + m, j] = w @ vh
    return dict(out=out)
