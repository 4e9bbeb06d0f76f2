"""What is measured of the 4-bit K/V cache: writing pages, appending tokens, reading pages back, and the
block-sparse retrieval decode step over them.

A slab holds one (page, kv head): 128 tokens of keys and values as 4-bit codes with a scale and a minimum
for each row (token).  For a row x of d values

    lo = min x,   scale = (max x - lo) / 15 rounded up to bf16,   code = rint((x - lo) / scale),

and the row stands for lo + code * scale; a constant row has scale 0.  Bytes of a slab: keys' codes
[128][d / 8] words (element 8 i + j of a token in word i), values' codes [4][d / 4][4][4] words (token
32 w + 8 t + j of element 4 c + e in word (w, c, t, e)), then keys' and values' rows [128] as (scale, lo)
in bf16.  The eight codes of a word sit at bits 4 (j / 2) + 16 (j mod 2).

The plain forms are elementary torch operations in 32 bits (64 for the scores, whose order decides which
blocks are kept).
"""
import math
import random

import torch

own = False

S = 128  # tokens a page
DEV = "cuda"
NIBBLES = (0, 16, 4, 20, 8, 24, 12, 28)  # the bit that code j of a word starts at


# ---- cases --------------------------------------------------------------------------------------------

def listed():
    return [
        # a 4096-token prompt of one layer (8 kv heads, d 128) compressed after prefill, and read back
        dict(name="pages prompt 4096", kind="pages", heads=8, d=128, pages=32, spare=0),
        # 4 requests x 131072 tokens of one layer compressed at once
        dict(name="pages 4x131072", kind="pages", heads=8, d=128, pages=4096, spare=0),
        # a few pages of a small model with d 64, among others that stay as they are
        dict(name="pages odd d64", kind="pages", heads=3, d=64, pages=37, spare=11),
        # the pages of a 16384-token shared prefix read back into bf16, as for the shared-prefix kernels
        dict(name="read back prefix 16384", kind="read", heads=8, d=128, pages=128, spare=3),
        # a 4 x 65536 cache read back
        dict(name="read back 4x65536 d64", kind="read", heads=8, d=64, pages=2048, spare=0),
        # one request's new token in a decode loop, in the middle of its page
        dict(name="append 1", kind="append", heads=8, d=128, batch=1, lo=65499, hi=65499),
        # a serving batch's new tokens, every request at another row of its page
        dict(name="append 64 ragged", kind="append", heads=8, d=128, batch=64, lo=2048, hi=8192),
        # one request below the dense boundary: every block is attended
        dict(name="decode 1x4096", kind="decode", q_heads=32, heads=8, d=128, batch=1, lo=4096, hi=4096,
             init=1024, local=7192, topk=0.2, boundary=32768),
        # the 65536-token layer
        dict(name="decode 1x65536", kind="decode", q_heads=32, heads=8, d=128, batch=1, lo=65536, hi=65536,
             init=1024, local=7192, topk=0.2, boundary=32768),
        # batch 4 x 131072, a fifth of the blocks
        dict(name="decode 4x131072", kind="decode", q_heads=32, heads=8, d=128, batch=4, lo=131072, hi=131072,
             init=1024, local=7192, topk=0.2, boundary=32768),
        # the same, every block: the largest read
        dict(name="decode 4x131072 dense", kind="decode", q_heads=32, heads=8, d=128, batch=4, lo=131072,
             hi=131072, init=1024, local=7192, topk=1.0, boundary=32768),
        # short and long requests together, empty ones and odd bounds among them, d 64
        dict(name="decode 13 ragged d64", kind="decode", q_heads=15, heads=5, d=64, batch=13, lo=0, hi=30000,
             init=300, local=1111, topk=0.33, boundary=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("pages", "read", "append", "decode", "decode", "decode"))
    d = rng.choice((64, 128))
    heads = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if kind in ("pages", "read"):
        most = 4096 * 8 // heads if kind == "pages" else 2048
        pages = _log(rng, 1, min(4096, most))
        return dict(kind=kind, heads=heads, d=d, pages=pages, spare=rng.randrange(0, 20))
    if kind == "append":
        hi = _log(rng, 128, 16384)
        return dict(kind=kind, heads=heads, d=d, batch=_log(rng, 1, 128), lo=rng.randrange(0, hi), hi=hi)
    group = rng.choice((1, 2, 3, 4, 5, 8))
    batch = _log(rng, 1, 24)
    hi = _log(rng, 128, min(131072, 4 * 131072 * 4 // (batch * heads)))
    lo = rng.choice((0, hi // 2, hi))
    topk = rng.choice((0.05, 0.1, 0.2, 0.35, 0.5))
    return dict(kind=kind, q_heads=group * heads, heads=heads, d=d, batch=batch, lo=lo, hi=hi,
                init=rng.choice((0, 64, 100, 256, 1024)), local=rng.choice((50, 128, 1000, 2048, 7192)), topk=topk,
                boundary=rng.choice((0, 8192, 32768)))


def _lens(case):
    """The requests' lengths: evenly from lo to hi, odd steps between."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _blocks(case, L):
    """(candidates, kept) of a request of L tokens."""
    W = L - case["local"]
    n = -(-W // S) - case["init"] // S if W > case["init"] else 0
    dense = L < case["boundary"]
    return n, (n if dense else min(n, max(0, math.ceil(case["topk"] * n - 1e-9))))


def _attended(case, L):
    """Tokens of a request that its heads attend (a kept block at the range's end counts whole)."""
    n, k = _blocks(case, L)
    W = L - case["local"]
    outside = L if W <= case["init"] else case["init"] + case["local"]
    return min(L, outside + k * S)


def work(case):
    d, H = case["d"], case["heads"]
    row = d + 8  # keys and values of one token: two rows of d / 2 bytes of codes and 4 of scale and minimum
    if case["kind"] == "pages":  # bf16 read, slabs written, bf16 written
        rows = case["pages"] * H * S
        return dict(bytes=rows * (4 * d + row + 4 * d), flops=rows * 2 * d * 6)
    if case["kind"] == "read":
        rows = case["pages"] * H * S
        return dict(bytes=rows * (row + 4 * d), flops=rows * 2 * d * 2)
    lens = _lens(case)
    if case["kind"] == "append":  # new rows in; codes and vectors out; the keys of each page read, the page read back
        rows = sum(L % S + 1 for L in lens) * H
        B = case["batch"] * H
        return dict(bytes=B * (4 * d + row + 4 * d) + rows * (d // 2 + 4) + B * S * (row + 4 * d),
                    flops=rows * d * 2 + B * S * 2 * d * 2)
    G = case["q_heads"] // H
    att = sum(_attended(case, L) for L in lens) * H
    cand = sum(n for n, k in (_blocks(case, L) for L in lens) if 0 < k < n) * H
    return dict(bytes=att * row + cand * d * 4 + case["batch"] * case["q_heads"] * d * 4,
                flops=att * 4 * G * d + cand * 2 * d)


# ---- the format in plain form ---------------------------------------------------------------------------

def _codes(x):
    """Rows x (fp32, holding bf16 values) as codes (int32), scale and minimum (bf16)."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo).double() / 15).float()  # in 64 bits: a quotient that bf16 holds must not come out above it
    scale = ((scale.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)  # up to bf16
    # the quotient in 64 bits: next to a half, 32 bits would round it onto the half
    code = torch.round((x - lo).double() / torch.where(scale > 0, scale, 1.0).double())
    return code.clamp_(max=15).int(), scale.bfloat16(), lo.bfloat16()


def _words(codes):
    """[..., 8] codes as words."""
    shifts = torch.tensor(NIBBLES, device=codes.device)
    return (codes.long() << shifts).sum(-1).int()


def _pack(k, v):
    """Keys and values [..., 128, d] (fp32) as slabs [..., bytes]."""
    d, lead = k.shape[-1], k.shape[:-2]
    (kc, ks, kl), (vc, vs, vl) = _codes(k), _codes(v)
    kw = _words(kc.reshape(*lead, S, d // 8, 8))
    n = len(lead)
    vw = vc.reshape(*lead, 4, 4, 8, d // 4, 4).permute(*range(n), n, n + 3, n + 1, n + 4, n + 2)
    vw = _words(vw)
    rows = [torch.cat((s, m), -1).contiguous() for s, m in ((ks, kl), (vs, vl))]
    return torch.cat([t.reshape(*lead, -1).contiguous().view(torch.uint8) for t in (kw, vw, *rows)], -1)


def _split(slabs, d):
    """Slabs [..., bytes] as key codes, value codes [..., 128, d] and rows (scale, minimum) [..., 128] in fp32."""
    lead, n = slabs.shape[:-1], slabs.dim() - 1
    shifts = torch.tensor(NIBBLES, device=slabs.device, dtype=torch.int32)

    def part(at, count, as_type):
        return slabs[..., at:at + count].contiguous().view(as_type)

    kc = (part(0, 64 * d, torch.int32).unsqueeze(-1) >> shifts) & 15
    vc = (part(64 * d, 64 * d, torch.int32).reshape(*lead, 4, d // 4, 4, 4, 1) >> shifts) & 15
    vc = vc.permute(*range(n), n, n + 2, n + 4, n + 1, n + 3)
    kr, vr = (part(at, 4 * S, torch.bfloat16).reshape(*lead, S, 2).float() for at in (128 * d, 128 * d + 4 * S))
    return (kc.reshape(*lead, S, d), vc.reshape(*lead, S, d), kr[..., 0], kr[..., 1], vr[..., 0], vr[..., 1])


def _values(slabs, d):
    kc, vc, ks, kl, vs, vl = _split(slabs, d)
    return (torch.addcmul(kl.unsqueeze(-1), kc.float(), ks.unsqueeze(-1)),
            torch.addcmul(vl.unsqueeze(-1), vc.float(), vs.unsqueeze(-1)))


def _slab_bytes(d):
    return S * d + 8 * S


def _rows_of(slabs, d):
    """The scales and minima of slabs, [..., K and V][128][2] in bf16: a view of the last 1024 bytes."""
    return slabs[..., S * d:].view(torch.bfloat16)


# ---- inputs ---------------------------------------------------------------------------------------------

def _random_pages(g, pages, heads, d):
    """Keys with a gain and an offset for each channel, as projections with a rotation leave them, and values."""
    gain = torch.rand(heads, 1, d, generator=g, device=DEV) + 0.5
    shift = torch.randn(heads, 1, d, generator=g, device=DEV) * 0.5
    k = (torch.randn(pages, heads, S, d, generator=g, device=DEV) * gain + shift).bfloat16()
    return k, torch.randn(pages, heads, S, d, generator=g, device=DEV).bfloat16()


def _slabs(g, pages, heads, d):
    """A cache of random slabs, and the keys' means."""
    kv = torch.empty(pages, heads, _slab_bytes(d), dtype=torch.uint8, device=DEV)
    reps = torch.empty(pages, heads, d, device=DEV)
    for p in range(0, pages, 256):
        k, v = _random_pages(g, min(256, pages - p), heads, d)
        kv[p:p + 256] = _pack(k.float(), v.float())
        reps[p:p + 256] = k.float().mean(2)
    return kv, reps


def _config(case):
    return dict(num_q_heads=case.get("q_heads", case["heads"]), num_kv_heads=case["heads"], head_dim=case["d"],
                block_size=S, init_tokens=case.get("init", 1024), local_tokens=case.get("local", 7192),
                topk_percent=case.get("topk", 0.2), dense_boundary=case.get("boundary", 32768), dtype=0)


def _permutation(g, n):
    return torch.randperm(n, generator=g, device=DEV).int()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind, H, d = case["kind"], case["heads"], case["d"]
    st = dict(case=case, cfg=_config(case), d=d)
    if kind in ("pages", "read"):
        n, total = case["pages"], case["pages"] + case["spare"]
        st["ids"], st["to"] = _permutation(g, total)[:n].contiguous(), _permutation(g, total)[:n].contiguous()
        st["k_out"], st["v_out"] = (torch.zeros(total, H, S, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")
        if kind == "read":
            st["kv"] = _slabs(g, total, H, d)[0]
        else:
            st["k"], st["v"] = (torch.empty(total, H, S, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")
            for p in range(0, total, 256):
                st["k"][p:p + 256], st["v"][p:p + 256] = _random_pages(g, min(256, total - p), H, d)
            st["kv"] = torch.zeros(total, H, _slab_bytes(d), dtype=torch.uint8, device=DEV)
        return st
    lens = _lens(case)
    B = len(lens)
    grown = [L + (kind == "append") for L in lens]
    blocks = [-(-L // S) for L in grown]
    nb = max(1, max(blocks))
    if kind == "append":  # only the pages that the new tokens go to exist twice over: the table names them alone
        st["tail"] = _permutation(g, B)
        table = torch.zeros(B, nb, dtype=torch.int32)
        for r, L in enumerate(lens):
            table[r, L // S] = st["tail"][r].item()
        pages = B
    else:
        pages = max(1, sum(blocks))
        perm = _permutation(g, pages).cpu()
        table, at = torch.full((B, nb), -1, dtype=torch.int32), 0
        for r, n in enumerate(blocks):
            table[r, :n] = perm[at:at + n]
            at += n
    st["table"] = table.to(DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["kv"], st["reps"] = _slabs(g, pages, H, d)
    if kind == "append":
        st["k_new"], st["v_new"] = (x[:, :, 0].contiguous() for x in _random_pages(g, B, H, d))
        st["order"] = torch.arange(B, dtype=torch.int32, device=DEV)
        st["k_out"], st["v_out"] = (torch.zeros(B, H, S, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")
        return st
    Hq = case["q_heads"]
    st["q"] = torch.randn(B, Hq, d, generator=g, device=DEV).bfloat16()
    _part_the_border(st, case, lens)
    kept = max(_blocks(case, nb * S)[1], max(_blocks(case, L)[1] for L in lens))
    if case["boundary"] > 0:
        kept = _blocks(case, nb * S)[0]
    st["kmax"] = max(1, kept)
    # blocks that a unit attends at most: the plain form gathers no more
    st["most"] = max(1, max(min(n, -(-min(case["init"], L) // S) + _blocks(case, L)[1] + min(n, case["local"] // S + 2))
                            for n, L in zip(blocks, lens)))
    st["sel"] = torch.full((B, H, st["kmax"]), -1, dtype=torch.int32, device=DEV)
    st["nsel"] = torch.zeros(B, H, dtype=torch.int32, device=DEV)
    st["out"] = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device=DEV)
    if own:
        from block_sparse_retrieval_gb300 import srkv
        st["workspace"] = torch.empty(srkv.decode_workspace_size(st["cfg"], B), dtype=torch.uint8, device=DEV)
    return st


def _part_the_border(st, case, lens):
    """Lifts the kept blocks' vectors by a thousandth of the scores' spread along the query: which blocks are kept
    then does not hang on the last bits of a 32-bit score."""
    H, G = case["heads"], case["q_heads"] // case["heads"]
    qsum = st["q"].double().reshape(len(lens), H, G, -1).sum(2)
    b_lo = case["init"] // S
    for r, L in enumerate(lens):
        n, k = _blocks(case, L)
        if not 0 < k < n:
            continue
        pages = st["table"][r, b_lo:b_lo + n].long()
        s = torch.einsum("nhd,hd->hn", st["reps"][pages].double(), qsum[r])
        lift = 1e-3 * s.std(1, keepdim=True) if n > 1 else s
        up = torch.zeros_like(s).scatter_(1, s.topk(k, 1).indices, 1.0) * lift
        st["reps"][pages] += torch.einsum("hn,hd->nhd", up, qsum[r] / qsum[r].square().sum(-1, keepdim=True)).float()


# ---- one pass -------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"pages": _plain_pages, "read": _plain_read, "append": _plain_append, "decode": _plain_decode}[st["case"]["kind"]](st)


def _own(st):
    from block_sparse_retrieval_gb300 import srkv
    kind, cfg, d = st["case"]["kind"], st["cfg"], st["d"]
    if kind == "pages":
        srkv.quantize_kv_int4(cfg, st["k"], st["v"], st["ids"], st["kv"], st["to"])
        srkv.dequantize_kv_int4(cfg, st["kv"], st["to"], st["k_out"], st["v_out"])
        return dict(k=st["k_out"], v=st["v_out"], rows=_rows_of(st["kv"], d))
    if kind == "read":
        srkv.dequantize_kv_int4(cfg, st["kv"], st["ids"], st["k_out"], st["v_out"], st["to"])
        return dict(k=st["k_out"], v=st["v_out"])
    if kind == "append":
        srkv.append_kv_int4(cfg, st["k_new"], st["v_new"], st["kv"], st["table"], st["lens"], st["reps"])
        srkv.dequantize_kv_int4(cfg, st["kv"], st["tail"], st["k_out"], st["v_out"], st["order"])
        return dict(k=st["k_out"], v=st["v_out"], rows=_rows_of(st["kv"], d), reps=st["reps"])
    srkv.retrieval_decode_int4(cfg, st["q"], st["kv"], st["reps"], st["table"], st["lens"], None, st["sel"],
                               st["nsel"], st["out"], st["workspace"])
    return dict(out=st["out"], sel=st["sel"], nsel=st["nsel"])


def _plain_pages(st):
    ids, to, d = st["ids"].long(), st["to"].long(), st["d"]
    st["kv"][to] = _pack(st["k"][ids].float(), st["v"][ids].float())
    k, v = _values(st["kv"][to], d)
    st["k_out"][to], st["v_out"][to] = k.bfloat16(), v.bfloat16()
    return dict(k=st["k_out"], v=st["v_out"], rows=_rows_of(st["kv"], d))


def _plain_read(st):
    k, v = _values(st["kv"][st["ids"].long()], st["d"])
    st["k_out"][st["to"].long()], st["v_out"][st["to"].long()] = k.bfloat16(), v.bfloat16()
    return dict(k=st["k_out"], v=st["v_out"])


def _plain_append(st):
    d, L = st["d"], st["lens"].long()
    page = st["table"].gather(1, (L // S).unsqueeze(1)).squeeze(1).long()
    kc, vc, ks, kl, vs, vl = _split(st["kv"][page], d)
    r = torch.arange(len(L), device=L.device)
    for code, scale, lo, new in ((kc, ks, kl, st["k_new"]), (vc, vs, vl, st["v_new"])):
        c, s, m = _codes(new.float())
        code[r, :, L % S], scale[r, :, L % S], lo[r, :, L % S] = c, s[..., 0].float(), m[..., 0].float()
    k = torch.addcmul(kl.unsqueeze(-1), kc.float(), ks.unsqueeze(-1))
    v = torch.addcmul(vl.unsqueeze(-1), vc.float(), vs.unsqueeze(-1))
    held = torch.arange(S, device=L.device) <= (L % S).unsqueeze(1)
    st["reps"][page] = torch.where(held[:, None, :, None], k, 0).sum(2) / (L % S + 1).view(-1, 1, 1)
    kw, n = _words(kc.reshape(*kc.shape[:2], S, d // 8, 8)), 2
    vw = _words(vc.reshape(*vc.shape[:2], 4, 4, 8, d // 4, 4).permute(0, 1, n, n + 3, n + 1, n + 4, n + 2))
    rows = [torch.stack((s, m), -1).bfloat16() for s, m in ((ks, kl), (vs, vl))]
    st["kv"][page] = torch.cat([t.reshape(*kc.shape[:2], -1).contiguous().view(torch.uint8) for t in (kw, vw, *rows)], -1)
    tail = torch.argsort(st["tail"].long())  # the pages, by their number, go out in the requests' order
    st["k_out"][tail[page]], st["v_out"][tail[page]] = k.bfloat16(), v.bfloat16()
    return dict(k=st["k_out"], v=st["v_out"], rows=_rows_of(st["kv"], d), reps=st["reps"])


def _plain_decode(st):
    c, d = st["case"], st["d"]
    B, H = st["nsel"].shape
    G = c["q_heads"] // H
    dev, NB = st["q"].device, st["table"].shape[1]
    L = st["lens"].long().view(B, 1, 1)
    W, table = L - c["local"], st["table"].long().clamp(min=0)
    b = torch.arange(NB, device=dev)
    # scores of the candidate blocks, and the k best, ties to the lower block
    q = st["q"].reshape(B, H, G, d)
    s = torch.einsum("bhd,bnhd->bhn", q.double().sum(2), st["reps"][table].double())
    cand = (torch.clamp(b * S, min=c["init"]) < torch.minimum(b * S + S, W)).expand(B, H, NB)
    n = cand.sum(-1, keepdim=True)
    k = torch.minimum(n, torch.ceil(c["topk"] * n.double() - 1e-9).clamp(min=0).long())
    k = torch.where(L < c["boundary"], n, k)
    order = torch.sort(torch.where(cand, s, -math.inf), dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(B, H, NB, dtype=torch.bool, device=dev).scatter_(2, order, b.expand(B, H, NB) < k)
    sel = torch.sort(torch.where(kept, b, NB), -1).values
    sel = torch.where(sel < NB, sel, -1)
    sel = torch.nn.functional.pad(sel, (0, max(0, st["kmax"] - NB)), value=-1)[..., :st["kmax"]].int()
    # the blocks with an attended token, gathered
    some = (kept | (b * S < c["init"]) | (b * S + S > W)) & (b * S < L)
    at = torch.sort(torch.where(some, b, NB), -1).values[..., :st["most"]]
    there, blk = at < NB, at.clamp(max=NB - 1)
    pages = table.unsqueeze(1).expand(B, H, NB).gather(2, blk)
    keys, vals = _values(st["kv"][pages, torch.arange(H, device=dev).view(1, H, 1)], d)
    tok = blk.unsqueeze(-1) * S + torch.arange(S, device=dev)
    L, W = L.unsqueeze(-1), W.unsqueeze(-1)
    mask = (tok < c["init"]) | (tok >= W) | (kept.gather(2, blk).unsqueeze(-1) & (tok >= c["init"]))
    mask = (mask & (tok < L) & there.unsqueeze(-1)).reshape(B, H, 1, -1)
    logit = torch.matmul(q.float(), keys.reshape(B, H, -1, d).transpose(-1, -2)) / math.sqrt(d)
    logit = torch.where(mask, logit, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vals.reshape(B, H, -1, d)) / torch.where(total > 0, total, 1.0)
    return dict(out=out.reshape(B, H * G, d).bfloat16(), sel=sel, nsel=k.expand(B, H, 1).squeeze(-1).int())


# ---- in 64 bits -----------------------------------------------------------------------------------------

def _exact_codes(x):
    """Codes, scale and minimum of rows in 64 bits: the scale is the next number of 8 significant bits upwards."""
    x = x.double()
    lo = x.min(-1, keepdim=True).values
    step = (x.max(-1, keepdim=True).values - lo) / torch.full_like(lo, 15.0)  # divided, not times 1 / 15
    m = torch.frexp(step).mantissa  # step / m is a power of two, exactly
    unit = torch.where(step == 0, torch.ones_like(step), step / m) / 256
    step = torch.ceil(step / unit) * unit
    c = torch.round((x - lo) / torch.where(step == 0, torch.ones_like(step), step))
    return torch.clamp(c, max=15.0), step, lo


def _exact_unpack(slab, d):
    """One (page, kv head) slab's rows in 64 bits, bit by bit: keys, values [128][d]."""
    w = slab.contiguous().view(torch.int32).long() & 0xFFFFFFFF
    nib = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1)  # [..., words, nibble]
    nib = nib[..., [0, 4, 1, 5, 2, 6, 3, 7]].double()
    lead = slab.shape[:-1]
    k = nib[..., :16 * d, :].reshape(*lead, S, d)
    v = torch.empty_like(k)
    vw = nib[..., 16 * d:32 * d, :].reshape(*lead, 4, d // 4, 4, 4, 8)
    for a in range(4):
        for t in range(4):
            for j in range(8):
                v[..., 32 * a + 8 * t + j, :] = vw[..., a, :, t, :, j].reshape(*lead, d)
    rows = slab[..., S * d:].contiguous().view(torch.bfloat16).double().reshape(*lead, 2, S, 2)
    return (k * rows[..., 0, :, :1] + rows[..., 0, :, 1:], v * rows[..., 1, :, :1] + rows[..., 1, :, 1:])


def exact(case, seed):
    st = prepare(case, seed)
    kind, d = case["kind"], case["d"]
    if kind == "pages":
        out = dict(k=torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV),
                   v=torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV))
        rows = torch.zeros(*st["k"].shape[:2], 2, S, 2, dtype=torch.float64, device=DEV)
        for at in range(0, len(st["ids"]), 256):
            a, b = st["ids"][at:at + 256].long(), st["to"][at:at + 256].long()
            for i, name in enumerate("kv"):
                c, step, lo = _exact_codes(st[name][a])
                out[name][b] = lo + c * step
                rows[b, :, i] = torch.cat((step, lo), -1)
        return dict(out, rows=rows.reshape(*rows.shape[:2], -1))
    if kind == "read":
        out = dict(k=torch.zeros(st["k_out"].shape, dtype=torch.float64, device=DEV),
                   v=torch.zeros(st["k_out"].shape, dtype=torch.float64, device=DEV))
        for at in range(0, len(st["ids"]), 256):
            a, b = st["ids"][at:at + 256].long(), st["to"][at:at + 256].long()
            out["k"][b], out["v"][b] = _exact_unpack(st["kv"][a], d)
        return out
    lens = st["lens"].tolist()
    if kind == "append":
        k, v = (torch.zeros(st["k_out"].shape, dtype=torch.float64, device=DEV) for _ in "kv")
        reps = st["reps"].double()
        rows = st["kv"][..., S * d:].contiguous().view(torch.bfloat16).double().reshape(len(lens), -1, 2, S, 2)
        for r, L in enumerate(lens):
            page, at = int(st["table"][r, L // S]), L % S
            both = _exact_unpack(st["kv"][page], d)
            place = int((st["tail"] == page).nonzero()[0, 0])
            for i, (old, new) in enumerate(zip(both, (st["k_new"][r], st["v_new"][r]))):
                c, step, lo = _exact_codes(new)
                old[:, at] = lo + c * step
                rows[page, :, i, at] = torch.cat((step, lo), -1)
                (k, v)[i][place] = old
            reps[page] = both[0][:, :at + 1].sum(1) / (at + 1)
        return dict(k=k, v=v, rows=rows.reshape(len(lens), rows.shape[1], -1), reps=reps)
    B, H, G = len(lens), case["heads"], case["q_heads"] // case["heads"]
    out = torch.zeros(B, case["q_heads"], d, dtype=torch.float64, device=DEV)
    sel, nsel = torch.full_like(st["sel"], -1), torch.zeros_like(st["nsel"])
    b_lo = case["init"] // S
    for r, L in enumerate(lens):
        n, k = _blocks(case, L)
        nb, W = -(-L // S), L - case["local"]
        pages = st["table"][r, :nb].long()
        for h in range(H if L else 0):
            q = st["q"][r, h * G:(h + 1) * G].double()
            s = st["reps"][pages[b_lo:b_lo + n], h].double() @ q.sum(0)
            best = sorted(range(n), key=lambda i, v=s.tolist(): (-v[i], i))[:k]
            kept = torch.tensor(sorted(best), dtype=torch.int64, device=DEV) + b_lo
            sel[r, h, :k], nsel[r, h] = kept.int(), k
            tok = torch.arange(nb * S, device=DEV)
            on = (tok < case["init"]) | (tok >= W)
            inside = torch.isin(tok // S, kept) & (tok >= case["init"]) & (tok < W)
            on = (on | inside) & (tok < L)
            need = on.view(nb, S).any(1)
            keys, vals = _exact_unpack(st["kv"][pages[need], h], d)
            on = on.view(nb, S)[need].reshape(-1)
            z = (q @ keys.reshape(-1, d)[on].T) / d ** 0.5
            p = torch.softmax(z, -1)
            out[r, h * G:(h + 1) * G] = p @ vals.reshape(-1, d)[on]
    return dict(out=out, sel=sel, nsel=nsel)
