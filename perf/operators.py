"""Cases of the paged 8-bit key/value cache: block tables and slot maps, the
append that quantises, the read-back, the decode and the chunked prefill over
the cache.

A page holds `block` tokens of every kv-head; each (page, head) has one scale
for its keys and one for its values.  Codes are e4m3 or int8, and a cached
value is code * scale.  `run` computes each operator in its plain form, or
calls the framework where `own` is true.
"""
import math

import torch

own = False

E4M3_MAX, INT8_MAX = 448.0, 127.0
BLOCK_HEADS = dict(Hq=32, Hkv=8, d=128, block=64)   # the shape of the repository's own decode workloads


def listed():
    return [
        # a batch of sequences that each generate one token: few new pages
        dict(name="tables_decode_step", op="tables", B=256, N=8192, block=64, grow=1, drop=0.02),
        # prompts arrive while others end: half a million slots
        dict(name="tables_prompts", op="tables", B=384, N=16384, block=64, grow=1500, drop=0.3),
        # the new token of 256 sequences goes into their caches, with its block's landmark
        dict(name="append_step", op="append", B=256, N=2048, grow=1, code="e4m3", **BLOCK_HEADS),
        # three ragged prompts are cached at once
        dict(name="append_prompts", op="append", B=3, N=16400, grow=14001, code="int8", **BLOCK_HEADS),
        # a short sequence is read back for the dense kernels
        dict(name="gather_short", op="gather", B=1, N=333, code="int8", **BLOCK_HEADS),
        # long sequences are read back
        dict(name="gather_long", op="gather", B=2, N=40000, code="e4m3", **BLOCK_HEADS),
        # one user, a short context: launch latency
        dict(name="decode_one", op="decode", B=1, N=200, top_k=0, code="e4m3", **BLOCK_HEADS),
        # the kept blocks of 64 long sequences (128K contexts, top-32 plus sink and local block), gated
        dict(name="decode_kept_128k", op="decode", B=64, N=131072, top_k=32, code="e4m3", **BLOCK_HEADS),
        # every block of ragged sequences, eight query heads per kv-head
        dict(name="decode_all_ragged", op="decode", B=32, N=32768, top_k=0, code="int8", Hq=32, Hkv=4, d=128, block=64),
        # a few drafted tokens of several sequences are verified at once
        dict(name="prefill_drafts", op="prefill", B=8, N=5000, grow=5, causal=True, code="int8", **BLOCK_HEADS),
        # the next chunk of two ragged prompts
        dict(name="prefill_chunk", op="prefill", B=2, N=9000, grow=1000, causal=True, code="e4m3", **BLOCK_HEADS),
        # a long chunk at the end of a 32K context
        dict(name="prefill_long", op="prefill", B=1, N=32768, grow=4096, causal=True, code="e4m3", **BLOCK_HEADS),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tables", "append", "gather", "decode", "prefill"])
    hkv = rng.choice([1, 2, 4, 8])
    heads = dict(Hq=hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=hkv, d=rng.choice([64, 128, 128, 128]),
                 block=rng.choice([16, 32, 64, 64, 64, 128]), code=rng.choice(["e4m3", "int8"]))
    if op == "tables":
        N = log(100, 16384)
        return dict(op=op, B=log(1, 384), N=N, block=heads["block"], grow=log(1, max(1, N // 8)), drop=rng.choice([0.0, 0.1, 0.3]))
    if op == "append":
        N = log(64, 14000)
        return dict(op=op, B=log(1, 24), N=N, grow=log(1, max(1, N // 8)), **heads)
    if op == "gather":
        return dict(op=op, B=log(1, 4), N=log(64, 20000), **heads)
    if op == "decode":
        N = log(64, 65536)
        return dict(op=op, B=log(1, max(1, min(64, 600000 // N))), N=N, top_k=rng.choice([0, 4, 16, 32]), **heads)
    N = log(64, 20000)
    return dict(op=op, B=log(1, max(1, min(8, 30000 // N))), N=N, grow=log(1, min(N, 2048)),
                causal=rng.random() < 0.75, **heads)


# ---- sizes --------------------------------------------------------------

def _lengths(case):
    """Lengths of the sequences: the first is N, the others spread below it."""
    N = case["N"]
    return [max(1, N - int(0.9 * N * ((b * 0.6180339887) % 1.0))) for b in range(case["B"])]


def _grown(case):
    """Tokens that each sequence has just gained (at most its length)."""
    lens = _lengths(case)
    return [max(1, min(n, case["grow"] - (case["grow"] // 3) * (b % 3) // 2)) for b, n in enumerate(lens)]


def _cap(case):
    return -(-case["N"] // case["block"])


def _is_dropped(case, b):
    """Whether sequence b ends in this step (its pages go back)."""
    return ((b * 0.7548776662) % 1.0) < case["drop"]


def work(case):
    op, bs = case["op"], case["block"]
    lens = _lengths(case)
    if op == "tables":
        grown = sum(g for b, g in enumerate(_grown(case)) if not _is_dropped(case, b))
        return {"bytes": 8 * grown + 12 * case["B"] + 8 * (grown // bs), "flops": 0}
    hkv, d, hq = case["Hkv"], case["d"], case["Hq"]
    if op == "append":
        new = sum(_grown(case))
        back = sum(len(r) for r in _touched(case))
        return {"bytes": new * hkv * d * (4 + 2) + back * hkv * d * (2 + 4), "flops": 0}
    if op == "gather":
        return {"bytes": sum(lens) * hkv * d * (2 + 4), "flops": 0}
    if op == "decode":
        if case["top_k"]:
            keys = sum(min(n, (min(case["top_k"] + 2, -(-n // bs)) - 1) * bs + (n - 1) % bs + 1) for n in lens)
        else:
            keys = sum(lens)
        return {"bytes": keys * hkv * d * 2 + case["B"] * hq * d * 4, "flops": 4.0 * keys * hq * d}
    pairs = sum(g * n - case["causal"] * g * (g - 1) // 2 for n, g in zip(lens, _grown(case)))
    return {"bytes": sum(lens) * hkv * d * 2 + sum(_grown(case)) * hq * (4 * d + 4), "flops": 4.0 * pairs * hq * d}


def _touched(case):
    """Positions of each sequence that lie in the blocks its new tokens go to."""
    bs = case["block"]
    return [range((n - g) // bs * bs, n) for n, g in zip(_lengths(case), _grown(case))]


# ---- inputs -------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _code_type(case):
    return torch.float8_e4m3fn if case["code"] == "e4m3" else torch.int8


def _codes(case, shape, g):
    """Codes of Gaussian values that nearly fill the code's range."""
    out = torch.empty(shape, dtype=_code_type(case), device="cuda")
    per = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], per):
        part = out[i:i + per]
        x = torch.randn(part.shape, generator=g, device="cuda")
        part.copy_(x.mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX) if case["code"] == "e4m3"
                   else x.mul_(32.0).round_().clamp_(-INT8_MAX, INT8_MAX))
    return out


def _cache(case, pages, g, power_of_two):
    """A filled cache: codes [pages, Hkv, block, d] and scales [pages, Hkv]."""
    shape = (pages, case["Hkv"], case["block"], case["d"])
    unit = 2.0 ** -7 if case["code"] == "e4m3" else 2.0 ** -5
    K, V = _codes(case, shape, g), _codes(case, shape, g)
    if power_of_two:
        ks, vs = (unit * 2.0 ** torch.randint(-1, 2, shape[:2], generator=g, device="cuda").float() for _ in "kv")
    else:
        ks, vs = (unit * (0.5 + torch.rand(shape[:2], generator=g, device="cuda")) for _ in "kv")
    return K, V, ks, vs


def _table(case, g):
    """A block table over shuffled pages; -1 behind a sequence's blocks."""
    lens, bs, cap = _lengths(case), case["block"], _cap(case)
    nb = torch.tensor([-(-n // bs) for n in lens])
    pages = int(nb.sum()) + 8
    held = torch.arange(cap)[None] < nb[:, None]
    table = torch.full((case["B"], cap), -1, dtype=torch.int32, device="cuda")
    table[held.cuda()] = torch.randperm(pages, generator=g, device="cuda")[:int(nb.sum())].int()
    return table, pages


def _params(case, pages, tokens, flags=0, top_k=0):
    import block_sparse_long_landmark_b200 as sa
    return sa.make_paged_params(case["B"], case.get("Hq", 1), case.get("Hkv", 1), case.get("d", 64), case["block"],
                                pages, _cap(case), tokens, top_k=top_k, flags=flags, code=case.get("code", "e4m3"))


def _slots(table, positions, bs):
    """Slots of the listed positions of each sequence, packed."""
    b = torch.cat([torch.full((len(r),), i) for i, r in enumerate(positions)]).cuda()
    pos = torch.cat([torch.arange(r.start, r.stop) for r in positions]).cuda()
    return table[b, pos // bs].long() * bs + pos % bs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, lens, bs = case["op"], _lengths(case), case["block"]
    s = dict(case=case, op=op, bs=bs)
    if op == "tables":
        old = [n - k for n, k in zip(lens, _grown(case))]
        new = [0 if _is_dropped(case, b) else n for b, n in enumerate(lens)]
        s["cur"], s["new"] = _i32(old), _i32(new)
        s["tokens"] = sum(max(0, n - o) for n, o in zip(new, old)) + 37
        cap = _cap(case)
        nb = torch.tensor([-(-n // bs) for n in old])
        pages = sum(-(-n // bs) for n in lens) + 8
        perm = torch.randperm(pages, generator=g, device="cuda").int()
        held = torch.arange(cap)[None] < nb[:, None]
        s["table"] = torch.full((case["B"], cap), -1, dtype=torch.int32, device="cuda")
        s["table"][held.cuda()] = perm[:int(nb.sum())]
        s["free"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["free"][:pages - int(nb.sum())] = perm[int(nb.sum()):]
        s["n_free"] = _i32([pages - int(nb.sum())])
        if own:
            s["p"] = _params(case, pages, s["tokens"])
    else:
        s["table"], pages = _table(case, g)
        s["len"] = _i32(lens)
        s["cache"] = _cache(case, pages, g, op == "append")
        tokens, flags, top_k = 0, 0, 0
        hq, hkv, d = case["Hq"], case["Hkv"], case["d"]
        if op in ("append", "prefill"):
            grown = _grown(case)
            s["cu"] = _i32([sum(grown[:b]) for b in range(case["B"] + 1)])
            tokens = sum(grown)
        if op == "append":
            s["slot"] = _slots(s["table"], [range(n - k, n) for n, k in zip(lens, grown)], bs)
            s["read"] = _slots(s["table"], _touched(case), bs)
            s["K"], s["V"] = (torch.randn(tokens, hkv, d, generator=g, device="cuda").bfloat16() for _ in "kv")
            s["L"] = torch.zeros(case["B"], hkv, _cap(case), d, dtype=torch.bfloat16, device="cuda")
        elif op == "gather":
            s["read"] = _slots(s["table"], [range(0, n) for n in lens], bs)
            tokens = sum(lens)
        elif op == "decode":
            s["q"] = torch.randn(case["B"], hq, d, generator=g, device="cuda").bfloat16()
            top_k = case["top_k"]
            if top_k:
                flags = 1 | 2 | 4 | 16          # sink, local block, gate, causal
                cap = top_k + 2
                nb = (s["len"] + bs - 1) // bs
                sc = torch.randn(case["B"], hkv, max(_cap(case), cap), generator=g, device="cuda")
                col = torch.arange(sc.shape[-1], device="cuda")
                rank = sc.masked_fill(col >= nb[:, None, None] - 1, -math.inf)
                rank = rank.masked_fill(col == 0, 1e9).masked_fill(col == nb[:, None, None] - 1, 1e9)
                best = rank.topk(cap, dim=-1)
                kept = torch.where(best.values > -math.inf, best.indices, 1 << 30).sort(-1).values
                held = kept < (1 << 30)
                s["count"] = held.sum(-1).int()
                s["idx"] = torch.where(held, kept, -1).int()
                s["score"] = torch.where(held, sc.gather(-1, torch.where(held, kept, 0)), 0.0).contiguous()
        else:
            s["Q"] = torch.randn(tokens, hq, d, generator=g, device="cuda").bfloat16()
            s["grown"], flags = max(grown), 16 if case["causal"] else 0
        if own:
            s["p"] = _params(case, pages, tokens, flags, top_k)
            if op == "append":
                s["p_read"] = _params(case, pages, s["read"].numel())
    if own:
        import block_sparse_long_landmark_b200 as sa
        s["ws"] = sa.paged_workspace(s["p"])
    return s


# ---- one pass -----------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_tables(s):
    import block_sparse_long_landmark_b200 as sa
    n_free, cu, slot = sa.paged_tables(s["p"], s["cur"], s["new"], s["free"], s["n_free"], s["table"], s["ws"])
    return {"table": s["table"], "free": s["free"], "n_free": n_free, "cu": cu, "slot": slot}


def _own_append(s):
    import block_sparse_long_landmark_b200 as sa
    sa.paged_append(s["p"], s["K"], s["V"], s["slot"], s["cache"], s["ws"], cu=s["cu"], new_len=s["len"], L=s["L"])
    K, V = sa.paged_gather(s["p_read"], s["read"], s["cache"], s["ws"])
    return {"K": K, "V": V, "L": s["L"]}


def _own_gather(s):
    import block_sparse_long_landmark_b200 as sa
    K, V = sa.paged_gather(s["p"], s["read"], s["cache"], s["ws"])
    return {"K": K, "V": V}


def _own_decode(s):
    import block_sparse_long_landmark_b200 as sa
    lists = (s["idx"], s["score"], s["count"]) if "idx" in s else None
    o, lse = sa.paged_decode(s["p"], s["q"], s["cache"], s["table"], s["len"], s["ws"], lists=lists)
    return {"o": o, "lse": lse}


def _own_prefill(s):
    import block_sparse_long_landmark_b200 as sa
    O, lse = sa.paged_prefill(s["p"], s["Q"], s["cu"], s["cache"], s["table"], s["len"], s["ws"])
    return {"O": O, "lse": lse}


def _plain_tables(s):
    """Pages of sequences that shrink are stacked on the free list; pages that
    are needed are popped from its top, in order of sequence and block."""
    bs, cur, new, table, free = s["bs"], s["cur"].long(), s["new"].long(), s["table"], s["free"]
    n_free = s["n_free"].long()
    b_old, b_new = (cur + bs - 1) // bs, (new + bs - 1) // bs
    n = (new - cur).clamp(min=0)
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    j = torch.arange(table.shape[1], device=table.device)
    back = (j >= b_new[:, None]) & (j < b_old[:, None])
    want = (j >= b_old[:, None]) & (j < b_new[:, None])
    R, A = back.sum(), want.sum()
    nth = (back.flatten().cumsum(0) - 1).view_as(back)
    P = free.numel()
    stack = torch.cat([free, free.new_zeros(P + 1)])
    stack[torch.where(back, n_free + nth, 2 * P)] = table
    top = n_free + R - 1 - (want.flatten().cumsum(0) - 1).view_as(want)
    table.copy_(torch.where(want, stack[top.clamp(0, 2 * P)], table))
    free.copy_(torch.where(torch.arange(P, device=free.device) < n_free + R - A, stack[:P], free))
    i = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp(max=len(n) - 1)
    pos = cur[b] + i - cu[b]
    slot = table[b, (pos // bs).clamp(max=table.shape[1] - 1)].long() * bs + pos % bs
    return {"table": table, "free": free, "n_free": (n_free + R - A).int(), "cu": cu.int(), "slot": torch.where(i < cu[-1], slot, -1)}


def _values(codes, scale):
    return codes.float() * scale[..., None, None]


def _rows(codes, page, off):
    """Rows `off` of the listed pages, every head: [T, Hkv, d] as fp32 codes."""
    return codes.view(torch.uint8)[page, :, off].view(codes.dtype).float()


def _quantised(case, codes, scales, x, page, nth, off, start, rows):
    """The touched pages after the append, codes as fp32 values and scales: a
    scale is kept while the new values fit, else it grows to the next power of
    two that holds them and the codes already there are rounded anew."""
    e4 = case["code"] == "e4m3"
    new = torch.zeros(len(page), *codes.shape[1:], device=x.device)
    new[nth, :, off] = x
    is_new = torch.zeros(len(page), codes.shape[2], dtype=torch.bool, device=x.device)
    is_new[nth, off] = True
    amax = new.abs().amax((2, 3))
    f, e = torch.frexp(amax)
    top, shift = (0.875, 9) if e4 else (0.9921875, 7)
    e = (e - shift + (f > top).int()).clamp(min=-126)
    had = (start > 0)[:, None]
    was = scales[page]
    fits = had & (amax <= was * (E4M3_MAX if e4 else INT8_MAX))
    power = ((e + 127) << 23).view(torch.float32)          # 2^e from its bits: pow() may be an ulp off
    now = torch.where(fits, was, power)
    old = codes.view(torch.uint8)[page].view(codes.dtype).float()
    ratio = torch.where(had, was / now, 1.0)[..., None, None]
    kept = (rows[None] < start[:, None])[:, None, :, None]
    y = torch.where(is_new[:, None, :, None], new / now[..., None, None], torch.where(kept, old * ratio, old))
    y = y.to(codes.dtype).float() if e4 else y.round()
    return y, now


def _plain_append(s):
    case, bs, slot = s["case"], s["bs"], s["slot"]
    K8, V8, ks, vs = s["cache"]
    page, nth = torch.unique(slot // bs, return_inverse=True)
    off = slot % bs
    rows = torch.arange(bs, device=slot.device)
    start = torch.full_like(page, bs).scatter_reduce(0, nth, off, "amin")
    last = torch.zeros_like(page).scatter_reduce(0, nth, off, "amax")
    k, now_k = _quantised(case, K8, ks, s["K"].float(), page, nth, off, start, rows)
    v, now_v = _quantised(case, V8, vs, s["V"].float(), page, nth, off, start, rows)
    K8.view(torch.uint8)[page] = k.to(K8.dtype).view(torch.uint8)
    V8.view(torch.uint8)[page] = v.to(V8.dtype).view(torch.uint8)
    ks[page], vs[page] = now_k, now_v
    # the landmark of each touched block: the mean of the cached keys
    i = torch.arange(len(slot), device=slot.device)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    blk = (s["len"].long()[b] - cu[b + 1] + i) // bs
    mean = torch.where((rows[None] <= last[:, None])[:, None, :, None], k, 0.0).sum(2) * now_k[..., None] / (last + 1)[:, None, None]
    s["L"][b, :, blk] = mean.to(s["L"].dtype)[nth]
    return {**_read(s), "L": s["L"]}


def _read(s):
    K8, V8, ks, vs = s["cache"]
    page, off = s["read"] // s["bs"], s["read"] % s["bs"]
    return {"K": (_rows(K8, page, off) * ks[page][..., None]).bfloat16(), "V": (_rows(V8, page, off) * vs[page][..., None]).bfloat16()}


def _plain_gather(s):
    return _read(s)


def _softmax_sum(z, v):
    """(softmax(z) v, log sum exp z); a row of -inf gives zeros and -inf."""
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m.clamp(min=-1e30)).exp_()
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l.clamp(min=1e-30), (m + l.log())[..., 0]


def _all_blocks(codes, scales, table):
    """Every cached row of the sequences: [B, Hkv, capacity, d] in fp32."""
    page = table.clamp(min=0).long()
    x = _values(codes.view(torch.uint8)[page].view(codes.dtype), scales[page])
    B, nb, H, bs, d = x.shape
    return x.transpose(1, 2).reshape(B, H, nb * bs, d)


def _plain_decode(s):
    case, bs = s["case"], s["bs"]
    K8, V8, ks, vs = s["cache"]
    B, H, d = case["B"], case["Hkv"], case["d"]
    q = s["q"].float().view(B, H, -1, d) / math.sqrt(d)
    if "idx" in s:
        blk = s["idx"].long()
        page = s["table"].long()[torch.arange(B, device=blk.device)[:, None, None], blk.clamp(min=0)]
        head = torch.arange(H, device=blk.device)[None, :, None]
        k = _values(K8.view(torch.uint8)[page, head].view(K8.dtype), ks[page, head]).flatten(2, 3)
        v = _values(V8.view(torch.uint8)[page, head].view(V8.dtype), vs[page, head]).flatten(2, 3)
        pos = (blk[..., None] * bs + torch.arange(bs, device=blk.device)).flatten(2)
        seen = (pos < s["len"][:, None, None]) & (blk[..., None] >= 0).expand(-1, -1, -1, bs).flatten(2)
        nb = (s["len"] + bs - 1)[:, None, None] // bs
        own_score = s["score"].gather(-1, (s["count"].long() - 1)[..., None])
        x = s["score"] - own_score
        gate = torch.where((blk == 0) | (blk == nb - 1), 0.0, torch.minimum(x, torch.zeros_like(x)) - torch.log1p(torch.exp(-x.abs())))
        bias = torch.where(seen, gate[..., None].expand(-1, -1, -1, bs).flatten(2), -math.inf)
    else:
        k, v = _all_blocks(K8, ks, s["table"]), _all_blocks(V8, vs, s["table"])
        pos = torch.arange(k.shape[2], device=k.device)
        bias = torch.where(pos < s["len"][:, None, None], 0.0, -math.inf)
    o, lse = _softmax_sum((q @ k.transpose(-1, -2)).add_(bias[:, :, None]), v)
    return {"o": o.reshape(B, -1, d).to(s["q"].dtype), "lse": lse.reshape(B, -1)}


def _plain_prefill(s):
    case = s["case"]
    K8, V8, ks, vs = s["cache"]
    B, H, d, T = case["B"], case["Hkv"], case["d"], s["grown"]
    k, v = _all_blocks(K8, ks, s["table"]), _all_blocks(V8, vs, s["table"])
    cu, n = s["cu"].long(), s["len"].long()
    own_row = torch.arange(T, device=cu.device)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + own_row).clamp(max=len(s["Q"]) - 1)                       # [B, T]
    q = s["Q"].float()[row].view(B, T, H, -1, d).permute(0, 2, 3, 1, 4) / math.sqrt(d)  # [B, H, G, T, d]
    z = q.reshape(B, H, -1, d) @ k.transpose(-1, -2)
    z = z.view(*q.shape[:4], k.shape[2])
    at = n[:, None] - count[:, None] + own_row
    if not case["causal"]:                # every key of the sequence, as to an encoder's states
        at = (n[:, None] - 1).expand_as(at)
    seen = torch.arange(k.shape[2], device=cu.device) <= at[..., None]
    z.masked_fill_(~seen[:, None, None], -math.inf)
    o, lse = _softmax_sum(z.view(B, H, -1, k.shape[2]), v)
    o = o.view(q.shape).permute(0, 3, 1, 2, 4).reshape(B, T, -1, d)
    lse = lse.view(q.shape[:4]).permute(0, 3, 1, 2).reshape(B, T, -1)
    is_row = own_row[None] < count[:, None]
    return {"O": o[is_row].to(s["Q"].dtype), "lse": lse[is_row]}


_own = dict(tables=_own_tables, append=_own_append, gather=_own_gather, decode=_own_decode, prefill=_own_prefill)
_plain = dict(tables=_plain_tables, append=_plain_append, gather=_plain_gather, decode=_plain_decode, prefill=_plain_prefill)


# ---- 64 bits ------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None                       # whole numbers only
    s = prepare(case, seed)
    return dict(append=_exact_append, gather=_exact_gather, decode=_exact_decode, prefill=_exact_prefill)[case["op"]](s)


def _exact_pages(codes, scales, pages):
    return torch.stack([codes[p].to(torch.float32).double() * scales[p].double()[:, None, None] for p in pages])


def _exact_read(s):
    out = []
    for codes, scales in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        flat = codes.transpose(1, 2).reshape(-1, *codes.shape[1:2], codes.shape[3])      # [slot, head, d]
        x = flat.view(torch.uint8)[s["read"]].view(codes.dtype).to(torch.float32).double()
        out.append(x * scales.double().repeat_interleave(s["bs"], 0)[s["read"]][..., None])
    return out


def _exact_gather(s):
    K, V = _exact_read(s)
    return {"K": K, "V": V}


def _power(e):
    """2^e for whole e in [-160, 160], exactly."""
    table = torch.tensor([math.ldexp(1.0, k) for k in range(-160, 161)], dtype=torch.float64, device=e.device)
    return table[e.long() + 160]


def _round_code(y, case):
    """Nearest code, ties to even: whole numbers, or three bits behind the
    leading one with steps of 2^-9 at the least."""
    if case["code"] == "int8":
        return y.round()
    step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(y / step) * step


def _exact_append(s):
    case, bs = s["case"], s["bs"]
    limit = E4M3_MAX if case["code"] == "e4m3" else INT8_MAX
    L = torch.zeros(s["L"].shape, dtype=torch.float64, device="cuda")
    lens, grown = _lengths(case), _grown(case)
    table = s["table"].tolist()
    back, at = {"K": [], "V": []}, 0
    for b, (n, k) in enumerate(zip(lens, grown)):
        first, t = (n - k) // bs * bs, n - k
        for lo in range(first, n, bs):
            hi, page = min(n, lo + bs), table[b][lo // bs]
            held = t - lo
            for name, codes, scales, x in (("K", s["cache"][0], s["cache"][2], s["K"]), ("V", s["cache"][1], s["cache"][3], s["V"])):
                fresh = x[at:at + hi - t].double().transpose(0, 1)               # [head, token, d]
                big = fresh.abs().amax((1, 2))
                need = torch.ceil(torch.log2(big / limit)).clamp(min=-126)
                need = need - (big <= limit * _power(need - 1)).double() + (big > limit * _power(need)).double()
                scale = _power(need.clamp(min=-126))
                was = scales[page].double()
                if held:
                    scale = torch.where(big <= was * limit, was, scale)
                new = _round_code(fresh / scale[:, None, None], case)
                old = codes[page, :, :held].to(torch.float32).double()
                old = _round_code(old * (was / scale)[:, None, None], case)
                vals = torch.cat([old, new], 1) * scale[:, None, None]
                back[name].append(vals.transpose(0, 1))
                if name == "K":
                    L[b, :, lo // bs] = vals.mean(1)
            at, t = at + hi - t, hi
    return {"K": torch.cat(back["K"]), "V": torch.cat(back["V"]), "L": L}


def _exact_attend(q, k, v, bias):
    """One head group: q [rows, d], k and v [keys, d], bias [rows, keys]."""
    z = q @ k.T / math.sqrt(q.shape[-1]) + bias
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def _exact_decode(s):
    case, bs = s["case"], s["bs"]
    B, hq, H, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    G, table, lens = hq // H, s["table"].tolist(), _lengths(case)
    o, lse = torch.zeros(B, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(B, hq, dtype=torch.float64, device="cuda")
    idx = s["idx"].tolist() if "idx" in s else None
    for b in range(B):
        every = list(range(-(-lens[b] // bs)))
        if idx is None:
            kb, vb = (_exact_pages(s["cache"][i], s["cache"][2 + i], [table[b][j] for j in every]) for i in (0, 1))
        for h in range(H):
            if idx is None:
                blocks, k, v = every, kb[:, h], vb[:, h]
            else:
                blocks = [j for j in idx[b][h] if j >= 0]
                pages = torch.tensor([table[b][j] for j in blocks], device="cuda")
                k, v = (s["cache"][i].view(torch.uint8)[pages, h].view(s["cache"][i].dtype).float().double() *
                        s["cache"][2 + i][pages, h].double()[:, None, None] for i in (0, 1))
            bias = torch.zeros(len(blocks), bs, dtype=torch.float64, device="cuda")
            bias[-1, lens[b] - blocks[-1] * bs:] = -math.inf
            if idx is not None:
                sc = s["score"][b, h, :len(blocks)].double()
                soft = -torch.nn.functional.softplus(-(sc - sc[-1]))
                inner = torch.tensor([0 < j < every[-1] for j in blocks], device="cuda")
                bias += torch.where(inner, soft, 0.0)[:, None]
            rows = slice(h * G, (h + 1) * G)
            o[b, rows], lse[b, rows] = _exact_attend(s["q"][b, rows].double(), k.reshape(-1, d), v.reshape(-1, d), bias.reshape(1, -1))
    return {"o": o, "lse": lse}


def _exact_prefill(s):
    case, bs = s["case"], s["bs"]
    hq, H, d = case["Hq"], case["Hkv"], case["d"]
    G, table = hq // H, s["table"].tolist()
    T = s["Q"].shape[0]
    O, lse = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, t) in enumerate(zip(_lengths(case), _grown(case))):
        k, v = (_exact_pages(s["cache"][i], s["cache"][2 + i], table[b][:-(-n // bs)]).transpose(0, 1).reshape(H, -1, d)[:, :n] for i in (0, 1))
        later = torch.arange(n, device="cuda") > torch.arange(n - t, n, device="cuda")[:, None]
        bias = torch.zeros(t, n, dtype=torch.float64, device="cuda")
        if case["causal"]:
            bias.masked_fill_(later, -math.inf)
        for h in range(hq):
            O[at:at + t, h], lse[at:at + t, h] = _exact_attend(s["Q"][at:at + t, h].double(), k[h // G], v[h // G], bias)
        at += t
    return {"O": O, "lse": lse}
