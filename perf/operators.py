"""What is measured of the 8-bit page cache: appends, attention, block-sparse attention and eviction.

The cache.  A page is 64 consecutive tokens of one KV head: int8 codes [64][D] for K and for V, one fp32 scale
for each (value = scale * code), and the smallest and largest K code of every channel over the tokens held.
Lists of page ids [S][Hk][capacity] and lengths [S] say which pages a sequence's heads read.

Operators.  "append" writes new tokens; "attn" attends over all pages of a list (with "mass": and adds each
page's attention weight to an accumulator); "sparse" picks blocks by an upper bound of their scores and attends
over the picked ones; "evict" keeps the pages of the largest accumulated weight and compacts the lists.
"""
import math
import random

import torch

own = False

PAGE = 64


# ------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's append: one new token for each of 32 running sequences, fp32 as the projections give it
        dict(name="append_token", op="append", S=32, nq=1, Hk=8, D=128, len=8192, ragged=True, x="f32"),
        # a prompt written in one call into lists that already hold an odd number of tokens
        dict(name="append_prompt", op="append", S=2, nq=4096, Hk=8, D=128, len=37, ragged=False, x="f16"),
        # the smallest decode call: one sequence, one token, 256 keys, where latency counts
        dict(name="attn_tiny", op="attn", S=1, nq=1, H=4, Hk=1, D=64, len=256, ragged=False, causal=False, out="f32", mass=False),
        # a decode step of eight sequences of different lengths (one of them empty)
        dict(name="attn_decode", op="attn", S=8, nq=1, H=32, Hk=8, D=128, len=32768, ragged=True, causal=False, out="f32", mass=False),
        # one sequence over a million keys, five query heads for each KV head
        dict(name="attn_long", op="attn", S=1, nq=1, H=40, Hk=8, D=128, len=1048576, ragged=False, causal=False, out="f16", mass=False),
        # a prompt's chunk of 512 tokens behind a long context
        dict(name="attn_prefill", op="attn", S=1, nq=512, H=32, Hk=8, D=128, len=32768, ragged=False, causal=True, out="f16", mass=False),
        # short chunks of eight sequences, results kept in fp32 to be merged with other partitions
        dict(name="attn_chunks", op="attn", S=8, nq=64, H=32, Hk=8, D=128, len=4096, ragged=True, causal=True, out="f32", mass=False),
        # sparse decode with a short context: 16 of 128 blocks
        dict(name="sparse_small", op="sparse", S=1, nq=1, H=32, Hk=8, D=128, len=8192, ragged=False, causal=False, out="f32", n_sel=16, n_first=1, n_last=1),
        # sparse decode over 262144 keys: 512 of 4096 blocks for each KV head
        dict(name="sparse_long", op="sparse", S=4, nq=1, H=32, Hk=4, D=128, len=262144, ragged=False, causal=False, out="f16", n_sel=512, n_first=1, n_last=2),
        # several queries a sequence (drafted tokens), each with its own blocks, ragged odd lengths
        dict(name="sparse_queries", op="sparse", S=2, nq=16, H=32, Hk=8, D=128, len=32747, ragged=True, causal=True, out="f16", n_sel=64, n_first=1, n_last=2),
        # a decode step that also accumulates each page's attention weight
        dict(name="attn_mass", op="attn", S=8, nq=1, H=32, Hk=8, D=128, len=32768, ragged=True, causal=False, out="f32", mass=True),
        # lists of about 2048 pages cut back to 512
        dict(name="evict", op="evict", S=8, Hk=8, len=131072, ragged=True, n_keep=512, n_first=1, n_last=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most_bytes = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["append", "attn", "attn", "attn", "sparse", "sparse", "evict"])
        S, D, Hk, G = _log(rng, 1, 32), rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 4, 5, 8])
        n, ragged = _log(rng, 1, 262144), rng.random() < 0.6
        if op == "append":
            c = dict(op=op, S=S, nq=_log(rng, 1, 4096), Hk=Hk, D=D, len=_log(rng, 1, 32768), ragged=ragged, x=rng.choice(["f32", "f16"]))
        elif op == "evict":
            keep = _log(rng, 6, 1024)
            c = dict(op=op, S=S, Hk=Hk, len=n, ragged=ragged, n_keep=keep, n_first=rng.randint(0, 2), n_last=rng.randint(1, 4))
        elif op == "sparse":
            nq = rng.choice([1, 1, 1, _log(rng, 1, 16)])
            c = dict(op=op, S=S, nq=nq, H=Hk * G, Hk=Hk, D=D, len=n, ragged=ragged, causal=nq > 1, out=rng.choice(["f32", "f16"]),
                     n_sel=_log(rng, 4, 512), n_first=rng.randint(0, 2), n_last=rng.randint(0, 2))
        else:
            nq = rng.choice([1, 1, _log(rng, 1, 1024)])
            c = dict(op=op, S=S, nq=nq, H=Hk * G, Hk=Hk, D=D, len=n, ragged=ragged, causal=nq > 1, out=rng.choice(["f32", "f16"]), mass=rng.random() < 0.3)
        w = work(c)
        pages = S * Hk * (n // PAGE + 2)
        rows = c["S"] * c.get("nq", 1) * c.get("H", 1)
        if w["bytes"] > most_bytes or w["flops"] > most_flops or (op in ("attn", "sparse") and rows * c["len"] > 1 << 29):
            continue
        if pages * PAGE * D * 2 > 2 << 30 or (op == "append" and c["nq"] * S * Hk * D > 1 << 23):
            continue
        if op == "sparse" and c["S"] * c["nq"] * Hk * min(c["n_sel"] * PAGE, n) * D > 1 << 30:
            continue
        return c


def _lens(c):
    """The sequences' lengths: all the same, or spread down to a fraction, the last of four or more empty."""
    S, n = c["S"], c["len"]
    if not c["ragged"]:
        return [n] * S
    lens = [max(1, n - (s * n * 7) // (8 * S)) for s in range(S)]
    if S >= 4 and c["op"] != "append":
        lens[-1] = 0
    return lens


def _pages(n):
    return -(-n // PAGE)


def work(c):
    lens = _lens(c)
    Hk = c["Hk"]
    if c["op"] == "append":
        D, n = c["D"], c["nq"]
        touched = sum(_pages(m + n) - m // PAGE for m in lens) * Hk
        x = 4 if c["x"] == "f32" else 2
        return {"bytes": c["S"] * n * Hk * D * 2 * (x + 1) + touched * (2 * 2 * D + 16 + 4), "flops": c["S"] * n * Hk * D * 4}
    if c["op"] == "evict":
        cap = _pages(max(lens)) + 2
        lists = c["S"] * Hk
        return {"bytes": sum(_pages(m) for m in lens) * Hk * 8 + lists * cap * 12, "flops": sum(_pages(m) for m in lens) * Hk}
    S, nq, H, D = c["S"], c["nq"], c["H"], c["D"]
    rows = S * nq * H
    ends = rows * (2 * D + (4 if c["out"] == "f32" else 2) * D + 4)
    seen = [[max(0, m - nq + t + 1) if c["causal"] else m for t in range(nq)] for m in lens]
    if c["op"] == "attn":
        keys = sum(lens) * Hk
        pages = sum(_pages(m) for m in lens) * Hk
        more = 8 * pages if c["mass"] else 0
        return {"bytes": keys * 2 * D + pages * 12 + ends + more, "flops": 4 * D * H * sum(map(sum, seen))}
    blocks = sum(_pages(m) for m in lens) * Hk
    picked = [[min(c["n_sel"], _pages(k)) * PAGE for k in row] for row in seen]
    # the pages that the queries of one sequence and head pick may be the same ones: what they cannot do without is one query's
    keys = sum(max(row) for row in picked) * Hk
    bytes_ = blocks * (2 * D + 8) + keys * 2 * D + keys // PAGE * 12 + ends + S * nq * Hk * c["n_sel"] * 4
    flops = 4 * D * H * sum(map(sum, picked)) + 4 * D * H * sum(_pages(k) for row in seen for k in row)
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------------------ the inputs

def _half(c):
    return torch.float32 if c["out"] == "f32" else torch.float16


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    lens = _lens(c)
    S, Hk = c["S"], c["Hk"]
    extra = c["nq"] if c["op"] == "append" else 0
    cap = _pages(max(lens) + extra) + 2
    held = [_pages(m + extra) for m in lens]
    n_pages = sum(held) * Hk + 5
    order = torch.randperm(n_pages, device=dev, generator=g).to(torch.int32)
    ids = torch.full((S, Hk, cap), -1, dtype=torch.int32, device=dev)
    at = 0
    for s in range(S):
        ids[s, :, : held[s]] = order[at : at + Hk * held[s]].view(Hk, held[s])
        at += Hk * held[s]
    st = dict(c=c, ids=ids, kv_len=torch.tensor(lens, dtype=torch.int32, device=dev))
    if c["op"] == "evict":
        # accumulated weights: a few pages hold most, many are near nothing, some were never looked at
        m = torch.rand((S, Hk, cap), device=dev, generator=g)
        m = (-torch.log(m.clamp_min(1e-6))) ** 3 * 0.05
        m[torch.rand(m.shape, device=dev, generator=g) < 0.2] = 0.0
        st["mass"] = m
        return st
    D = c["D"]
    k = torch.empty((n_pages, PAGE, D), dtype=torch.int8, device=dev)
    v = torch.empty((n_pages, PAGE, D), dtype=torch.int8, device=dev)
    step = max(1, (1 << 26) // (PAGE * D))
    for a in range(0, n_pages, step):
        n = min(step, n_pages - a)
        # keys of one block resemble each other: a direction of the block and each token's own part
        x = torch.randn((n, 1, D), device=dev, generator=g) * 18 + torch.randn((n, PAGE, D), device=dev, generator=g) * 24
        k[a : a + n] = x.round_().clamp_(-127, 127).to(torch.int8)
        x = torch.randn((n, PAGE, D), device=dev, generator=g) * 30
        v[a : a + n] = x.round_().clamp_(-127, 127).to(torch.int8)
    ks = torch.rand(n_pages, device=dev, generator=g) * 0.03 + 0.02
    vs = torch.rand(n_pages, device=dev, generator=g) * 0.03 + 0.01
    # what a page's last tokens are is left over from its last owner: the smallest and largest codes leave them out
    rows = torch.full((n_pages,), 0, dtype=torch.int32, device=dev)
    left = (st["kv_len"].view(S, 1, 1) - torch.arange(cap, device=dev, dtype=torch.int32) * PAGE).clamp(0, PAGE).expand(S, Hk, cap)
    rows[ids[ids >= 0].long()] = left[ids >= 0].to(torch.int32)
    lo = torch.zeros((n_pages, D), dtype=torch.int8, device=dev)
    hi = torch.zeros((n_pages, D), dtype=torch.int8, device=dev)
    for a in range(0, n_pages, step):
        on = torch.arange(PAGE, device=dev).view(1, PAGE, 1) < rows[a : a + step].view(-1, 1, 1)
        kk = k[a : a + step]
        lo[a : a + step] = torch.where(on, kk, 127).amin(1)
        hi[a : a + step] = torch.where(on, kk, -127).amax(1)
    empty = rows == 0
    lo[empty], hi[empty], ks[empty], vs[empty] = 0, 0, 0.0, 0.0
    st.update(k=k, v=v, ks=ks, vs=vs, lo=lo, hi=hi)
    if c["op"] == "append":
        t = torch.float32 if c["x"] == "f32" else torch.float16
        st["k_new"] = (torch.randn((S, c["nq"], Hk, D), device=dev, generator=g) * 1.1).to(t)
        st["v_new"] = torch.randn((S, c["nq"], Hk, D), device=dev, generator=g).to(t)
        return st
    st["q"] = torch.randn((S, c["nq"], c["H"], D), device=dev, generator=g).to(torch.float16)
    st["q_pos"] = None
    if c["causal"]:
        st["q_pos"] = (st["kv_len"].view(S, 1) - c["nq"] + torch.arange(c["nq"], device=dev, dtype=torch.int32)).to(torch.int32).contiguous()
    if c.get("mass"):
        st["mass"] = torch.rand((S, Hk, cap), device=dev, generator=g)
    return st


# --------------------------------------------------------------------------------------------- the operators

_handle = None


def _own(st):
    """The framework, its handle (kept by the program) and the pool over the state's tensors (kept with them)."""
    global _handle
    import split_kv_flash_attn_gb300 as skv
    if _handle is None:
        _handle = skv.Handle(torch.cuda.current_device())
    if "k" in st and "pool" not in st:
        st["pool"] = skv.Q8Pool(st["k"], st["v"], st["ks"], st["vs"], st["lo"], st["hi"])
    return skv, _handle


def run(st):
    return {"append": _append, "attn": _attn, "sparse": _sparse, "evict": _evict}[st["c"]["op"]](st)


def _append(st):
    # The codes come back as they are held: the rule that gives them is exact, so they have to be equal.
    out = {n: st[n] for n in ("k", "v", "ks", "vs", "lo", "hi")}
    if own:
        skv, h = _own(st)
        skv.q8_append(h, st["pool"], st["k_new"], st["v_new"], st["ids"], st["kv_len"])
        return out
    c, dev = st["c"], st["ids"].device
    S, n, Hk, D = st["k_new"].shape
    P = _pages(n + PAGE - 1)
    first = (st["kv_len"] // PAGE).view(S, 1, 1)
    blk = first + torch.arange(P, device=dev).view(1, 1, P)
    pos = blk.unsqueeze(-1) * PAGE + torch.arange(PAGE, device=dev)                       # [S,1,P,64]: the token of each row
    here = (pos < (st["kv_len"] + n).view(S, 1, 1, 1)).expand(S, Hk, P, PAGE)
    old = (pos < st["kv_len"].view(S, 1, 1, 1)).expand(S, Hk, P, PAGE)
    new = here & ~old
    page = st["ids"].gather(2, blk.clamp_max(st["ids"].shape[2] - 1).expand(S, Hk, P).long())
    on = new.any(-1)
    at = page[on].long()
    tok = (pos - st["kv_len"].view(S, 1, 1, 1)).clamp(0, n - 1).expand(S, Hk, P, PAGE)
    for x, codes, scale in ((st["k_new"], st["k"], st["ks"]), (st["v_new"], st["v"], st["vs"])):
        xs = x.permute(0, 2, 1, 3).float()                                                 # [S,Hk,n,D]
        xr = xs.gather(2, tok.reshape(S, Hk, P * PAGE, 1).expand(S, Hk, P * PAGE, D)).view(S, Hk, P, PAGE, D)[on]
        is_new, is_old = new[on].unsqueeze(-1), old[on].unsqueeze(-1)
        amax = torch.where(is_new, xr.abs(), 0.0).amax((1, 2))
        d0 = torch.where(is_old.any(1).view(-1), scale[at], 0.0)
        d1 = torch.maximum(d0, (amax.double() / 127.0).float())
        div = torch.where(d1 > 0, d1, 1.0).double().view(-1, 1, 1)
        c0 = codes[at]
        kept = (c0.double() * d0.double().view(-1, 1, 1) / div).round()
        put = (xr.double() / div).round().clamp(-127, 127)
        codes[at] = torch.where(is_new, put, torch.where(is_old, kept, c0.double())).to(torch.int8)
        scale[at] = d1
        if codes is st["k"]:
            is_here = is_new | is_old
            st["lo"][at] = torch.where(is_here, codes[at], 127).amin(1)
            st["hi"][at] = torch.where(is_here, codes[at], -127).amax(1)
    return out


def _attend(st, ids, seen, H):
    """Attention of q [S',nq,H,D] over whole lists ids [S',Hk,P]; seen [S',Hk,nq,P*64]: which keys a query sees."""
    q = st["q"].view(ids.shape[0], -1, H, st["q"].shape[-1])
    S, nq, _, D = q.shape
    Hk, P = ids.shape[1:]
    G = H // Hk
    page = ids.clamp_min(0).long()
    k = (st["k"][page].float() * st["ks"][page].view(S, Hk, P, 1, 1)).view(S, Hk, P * PAGE, D)
    qq = q.float().view(S, nq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hk, nq * G, D)
    s = (qq @ k.transpose(2, 3)).view(S, Hk, nq, G, P * PAGE) / math.sqrt(D)
    del k
    s = s.masked_fill_(~seen.unsqueeze(3), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + l.log(), -math.inf)
    p = p.div_(torch.where(l > 0, l, 1.0))
    v = (st["v"][page].float() * st["vs"][page].view(S, Hk, P, 1, 1)).view(S, Hk, P * PAGE, D)
    o = (p.view(S, Hk, nq * G, P * PAGE) @ v).view(S, Hk, nq, G, D)
    back = lambda x: x.permute(0, 2, 1, 3, 4).reshape(S, nq, H, -1)  # noqa: E731
    return back(o), back(lse).squeeze(-1), p


def _limit(st):
    """[S,nq]: how many keys each query sees."""
    n = st["kv_len"].view(-1, 1).expand(-1, st["q"].shape[1])
    return n if st["q_pos"] is None else torch.minimum(n, st["q_pos"] + 1)


def _attn(st):
    c = st["c"]
    if own:
        skv, h = _own(st)
        o, lse = skv.q8_attn(h, st["pool"], st["q"], st["ids"], st["kv_len"], q_pos=st["q_pos"], mass=st.get("mass"), o_dtype=_half(c))
        return (o, lse, st["mass"]) if c["mass"] else (o, lse)
    S, Hk, cap = st["ids"].shape
    P = _pages(max(_lens(c)))
    ids = st["ids"][:, :, :P]
    seen = torch.arange(P * PAGE, device=ids.device).view(1, 1, 1, -1) < _limit(st).view(S, 1, -1, 1)
    o, lse, p = _attend(st, ids, seen.expand(S, Hk, -1, -1), c["H"])
    if not c["mass"]:
        return o.to(_half(c)), lse
    st["mass"][:, :, :P] += p.sum((2, 3)).view(S, Hk, P, PAGE).sum(-1)
    return o.to(_half(c)), lse, st["mass"]


def _sparse(st):
    c = st["c"]
    if own:
        skv, h = _own(st)
        sel = skv.q8_select(h, st["pool"], st["q"], st["ids"], st["kv_len"], n_sel=c["n_sel"], n_first=c["n_first"], n_last=c["n_last"], q_pos=st["q_pos"])
        o, lse = skv.q8_attn(h, st["pool"], st["q"], st["ids"], st["kv_len"], q_pos=st["q_pos"], sel=sel, o_dtype=_half(c))
        return o, lse, sel
    S, nq, H, D = st["q"].shape
    Hk = c["Hk"]
    G = H // Hk
    P = _pages(max(_lens(c)))
    ids = st["ids"][:, :, :P]
    page = ids.clamp_min(0).long()
    # the query in 8 bits; rounding goes by the exact quotient, so that everybody picks the same blocks
    q = st["q"].float().view(S, nq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hk, nq * G, D)
    dq = (q.abs().amax(-1, keepdim=True).double() / 127.0).float()
    cq = (q.double() / torch.where(dq > 0, dq, 1.0).double()).round().clamp(-127, 127).float()
    # whole numbers below 2^24: the sums are exact in 32 bits
    dots = cq.clamp_min(0) @ st["hi"][page].float().transpose(2, 3) + cq.clamp_max(0) @ st["lo"][page].float().transpose(2, 3)
    bound = (dots * dq).view(S, Hk, nq, G, P).amax(3) * st["ks"][page].unsqueeze(2)        # [S,Hk,nq,P]
    blk = torch.arange(P, device=ids.device).view(1, 1, 1, P)
    limit = _limit(st)
    nb = ((limit.clamp_min(0) + PAGE - 1) // PAGE).view(S, 1, nq, 1)
    may = (blk < nb) & (ids >= 0).unsqueeze(2)
    must = may & ((blk < c["n_first"]) | (blk >= nb - c["n_last"]))
    rank = torch.where(must, math.inf, torch.where(may, bound, -math.inf))
    n = min(c["n_sel"], P)
    got, sel = torch.sort(rank, dim=-1, descending=True, stable=True)
    sel = torch.where(got[..., :n] > -math.inf, sel[..., :n], P).sort(-1).values
    sel = torch.where(sel < P, sel, -1).permute(0, 2, 1, 3)                                # [S,nq,Hk,n]
    full = torch.full((S, nq, Hk, c["n_sel"]), -1, dtype=torch.int32, device=ids.device)
    full[..., :n] = sel.to(torch.int32)
    # every query is a sequence of its own over its own list
    mine = ids.unsqueeze(1).expand(S, nq, Hk, P).gather(3, sel.clamp_min(0)).reshape(S * nq, Hk, n)
    pos = sel.clamp_min(0).unsqueeze(-1) * PAGE + torch.arange(PAGE, device=ids.device)
    seen = (pos < limit.view(S, nq, 1, 1, 1)) & (sel >= 0).unsqueeze(-1)
    o, lse, _ = _attend(st, mine, seen.reshape(S * nq, Hk, 1, n * PAGE), H)
    return o.view(S, nq, H, D).to(_half(c)), lse.view(S, nq, H), full


def _evict(st):
    c = st["c"]
    if own:
        skv, h = _own(st)
        return skv.q8_evict(h, st["ids"], st["mass"], st["kv_len"], n_keep=c["n_keep"], n_first=c["n_first"], n_last=c["n_last"])
    ids, mass, kv_len = st["ids"], st["mass"], st["kv_len"]
    S, Hk, cap = ids.shape
    blk = torch.arange(cap, device=ids.device).view(1, 1, cap)
    nb = ((kv_len + PAGE - 1) // PAGE).view(S, 1, 1)
    must = (blk < c["n_first"]) | (blk >= nb - c["n_last"])
    rank = torch.where(blk >= nb, -math.inf, torch.where(must, math.inf, torch.where(ids < 0, -1.0, mass)))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(2, order, blk.expand(S, Hk, cap).contiguous())
    keep = (place < c["n_keep"]) | (blk >= nb)                                             # pages behind the last token move along
    front = torch.sort(keep.to(torch.int8), dim=-1, descending=True, stable=True).indices
    n = keep.sum(-1, keepdim=True)
    out_ids = torch.where(blk < n, ids.gather(2, front), -1)
    out_mass = torch.where(blk < torch.minimum(nb, torch.tensor(c["n_keep"], device=ids.device)), mass.gather(2, front), 0.0)
    gone = torch.sort((~keep & (ids >= 0)).to(torch.int8), dim=-1, descending=True, stable=True).indices
    freed = torch.where(blk < (~keep & (ids >= 0)).sum(-1, keepdim=True), ids.gather(2, gone), -1)
    out_len = kv_len - (nb.view(S) - c["n_keep"]).clamp_min(0).to(torch.int32) * PAGE
    return out_ids, out_mass, out_len, freed


# --------------------------------------------------------------------------------- the definitions in 64 bits

def _list64(st, s, kh, blocks):
    """The keys and values of some blocks of one list, in 64 bits."""
    page = st["ids"][s, kh, blocks].long()
    k = st["k"][page].double() * st["ks"][page].double()[:, None, None]
    v = st["v"][page].double() * st["vs"][page].double()[:, None, None]
    return k.flatten(0, 1), v.flatten(0, 1)


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "evict":
        # list by list: a page's rank is its weight, with the first and the last ones above all others
        S, Hk, cap = st["ids"].shape
        ids, mass = st["ids"].cpu().tolist(), st["mass"].double().cpu()
        out = torch.zeros_like(mass)
        for s, n in enumerate(_lens(c)):
            nb = _pages(n)
            for kh in range(Hk):
                m = mass[s, kh].tolist()
                held = set(range(min(c["n_first"], nb))) | set(range(max(0, nb - c["n_last"]), nb))
                rest = sorted((b for b in range(nb) if b not in held), key=lambda b: (ids[s][kh][b] < 0, -m[b], b))
                kept = sorted(held | set(rest[: max(0, c["n_keep"] - len(held))]))
                out[s, kh, : len(kept)] = mass[s, kh, torch.tensor(kept, dtype=torch.long)]
        return None, out.to(st["mass"].device), None, None
    if c["op"] == "append":
        # scales from the largest magnitudes, taken from their definition page by page
        ks, vs = st["ks"].double().clone(), st["vs"].double().clone()
        n = c["nq"]
        for s, m in enumerate(_lens(c)):
            for b in range(m // PAGE, _pages(m + n)):
                lo, hi = max(b * PAGE, m), min((b + 1) * PAGE, m + n)
                page = st["ids"][s, :, b].long()
                for x, d in ((st["k_new"], ks), (st["v_new"], vs)):
                    top = x[s, lo - m : hi - m].double().abs().amax((0, 2)) / 127.0
                    d[page] = torch.maximum(d[page], top) if m > b * PAGE else top
        return {"k": None, "v": None, "ks": ks, "vs": vs, "lo": None, "hi": None}
    S, nq, H, D = st["q"].shape
    Hk, G, dev = c["Hk"], H // c["Hk"], st["q"].device
    o = torch.zeros((S, nq, H, D), dtype=torch.float64, device=dev)
    lse = torch.full((S, nq, H), -math.inf, dtype=torch.float64, device=dev)
    mass = st["mass"].double() if c.get("mass") else None
    if c["op"] == "sparse" and S * nq * Hk > 2048:
        return None
    for s, n in enumerate(_lens(c)):
        if n == 0:
            continue
        for kh in range(Hk):
            qh = st["q"][s, :, kh * G : (kh + 1) * G].double()                            # [nq,G,D]
            if c["op"] == "attn":
                k, v = _list64(st, s, kh, slice(0, _pages(n)))
                w = torch.einsum("tgd,jd->tgj", qh, k[:n]) * D ** -0.5
                if c["causal"]:
                    last = n - nq + torch.arange(nq, device=dev)
                    w.masked_fill_(torch.arange(n, device=dev)[None, None] > last[:, None, None], -math.inf)
                z = torch.logsumexp(w, -1)
                p = torch.where(z[..., None] > -math.inf, torch.exp(w - z.clamp_min(-1e300)[..., None]), 0.0)
                o[s, :, kh * G : (kh + 1) * G] = torch.einsum("tgj,jd->tgd", p, v[:n])
                lse[s, :, kh * G : (kh + 1) * G] = z
                if mass is not None:
                    pad = torch.zeros(_pages(n) * PAGE, dtype=torch.float64, device=dev)
                    pad[:n] = p.sum((0, 1))
                    mass[s, kh, : _pages(n)] += pad.view(-1, PAGE).sum(1)
                continue
            for t in range(nq):
                m = min(n, n - nq + t + 1) if c["causal"] else n
                if m <= 0:
                    continue
                nb = _pages(m)
                page = st["ids"][s, kh, :nb].long()
                top = qh[t].abs().amax(-1, keepdim=True)
                dq = (top / 127.0).float().double()
                code = torch.round(qh[t] / dq.clamp_min(1e-300)).clamp(-127, 127)
                lo, hi = st["lo"][page].double(), st["hi"][page].double()
                dots = torch.where(code[:, None] > 0, code[:, None] * hi[None], code[:, None] * lo[None]).sum(-1)
                # the bound is held in 32 bits: rounded after each of its two products
                score = ((dots * dq).float().amax(0).double() * st["ks"][page].double()).float()
                score[: c["n_first"]] = math.inf
                if c["n_last"]:
                    score[max(0, nb - c["n_last"]) :] = math.inf
                pick = torch.argsort(score, descending=True, stable=True)[: c["n_sel"]].sort().values
                k, v = _list64(st, s, kh, pick)
                far = (pick[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten() >= m
                w = (qh[t] @ k.T * D ** -0.5).masked_fill(far, -math.inf)
                z = torch.logsumexp(w, -1)
                o[s, t, kh * G : (kh + 1) * G] = torch.exp(w - z[:, None]) @ v
                lse[s, t, kh * G : (kh + 1) * G] = z
    if c["op"] == "attn":
        return (o, lse, mass) if c["mass"] else (o, lse)
    return o, lse, None
