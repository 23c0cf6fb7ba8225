"""What is measured of the rows around attention: norm and rotation of queries and keys, the cache rows they become,
and the gradients of both and of attention itself.

"rope": RMS norm of each head's query and key and the rotation by the token's positions.  "append": the same with the
keys and values written into cache rows.  "rope_back": gradients of "rope" for the rows and the norm's weights.
"attn_back": gradients of attention over a range of cache rows (or row lists) for queries, keys and values, from the
output, its log-sum-exp and the output's gradient.
"""
import math
import random

import torch

own = False

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = {"f32": F32, "f16": F16, "bf16": BF16}


# ------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one sequence with a single KV head: the smallest serving call, where latency counts
        dict(name="append_token", op="append", n=1, H=4, Hk=1, D=64, R=64, axes=1, pairs="half", norm=False, x="f16", far=4095, kt="f16", vt="f16"),
        # a decode step of 32 sequences, far into their contexts
        dict(name="append_decode", op="append", n=32, H=32, Hk=8, D=128, R=128, axes=1, pairs="half", norm=True, x="f16", far=131072, kt="f16", vt="f16"),
        # a prompt whose keys and values go to fp16 rows
        dict(name="append_prompt", op="append", n=4096, H=32, Hk=8, D=128, R=128, axes=1, pairs="half", norm=True, x="f16", far=0, kt="f16", vt="f16"),
        # a prompt chunk whose keys and values go to q8_0 and q4_0 rows; half of each head is rotated
        dict(name="append_quant", op="append", n=1021, H=32, Hk=8, D=128, R=64, axes=1, pairs="interleaved", norm=False, x="f32", far=65024, kt="q8_0", vt="q4_0"),
        # queries and keys of a training step's 8192 tokens
        dict(name="rope_train", op="rope", n=8192, H=32, Hk=8, D=128, R=128, axes=1, pairs="half", norm=True, x="f16", far=0, out="f16"),
        # the patches of an image: time, height and width, 71 x 71 of them, small heads
        dict(name="rope_image", op="rope", n=5041, H=16, Hk=16, D=64, R=64, axes=3, pairs="interleaved", norm=False, x="bf16", far=71, out="f32"),
        # the gradients of rope_train
        dict(name="rope_back_train", op="rope_back", n=8192, H=32, Hk=8, D=128, R=128, axes=1, pairs="half", norm=True, x="f16", far=0, out="f16"),
        # the gradients of a few hundred tokens with three axes, fp32 rows
        dict(name="rope_back_image", op="rope_back", n=611, H=16, Hk=16, D=64, R=64, axes=3, pairs="half", norm=True, x="f32", far=25, out="f32"),
        # the smallest training call: 64 tokens, small heads, one KV head
        dict(name="attn_back_tiny", op="attn_back", S=1, nq=64, n=256, H=4, Hk=1, D=64, causal=True, lists=False, part=0),
        # a chunk of 512 tokens at the end of 32768 keys
        dict(name="attn_back_chunk", op="attn_back", S=1, nq=512, n=32768, H=32, Hk=8, D=128, causal=True, lists=False, part=0),
        # a training step's batch of ragged sequences in one cache, by row lists
        dict(name="attn_back_batch", op="attn_back", S=4, nq=2048, n=2048, H=32, Hk=8, D=128, causal=True, lists=True, part=0),
        # one long sequence, causal
        dict(name="attn_back_long", op="attn_back", S=1, nq=16384, n=16384, H=8, Hk=2, D=128, causal=True, lists=False, part=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most_bytes = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["append", "rope", "rope_back", "attn_back", "attn_back", "attn_back"])
        D, Hk, G = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 4, 5, 8])
        if op == "attn_back":
            lists = rng.random() < 0.35
            S = _log(rng, 1, 8) if lists or rng.random() < 0.2 else 1
            nq, n = _log(rng, 1, 8192), _log(rng, 1, 65536)
            # a causal call's tokens are its last ones, or all that there are; a partition leaves the first `part` keys to another
            causal = rng.random() < 0.6
            if causal and rng.random() < 0.5:
                nq = n = min(nq, n)
            part = 0 if lists or rng.random() < 0.7 else rng.randint(0, n - 1)
            c = dict(op=op, S=S, nq=nq, n=n, H=Hk * G, Hk=Hk, D=D, causal=causal, lists=lists, part=part)
            if S * nq * Hk * G * n > 1 << 31 or S * n * Hk * D > 1 << 27:
                continue
        else:
            R = rng.choice([D, D, D // 2])
            c = dict(op=op, n=_log(rng, 1, 8192), H=Hk * G, Hk=Hk, D=D, R=R, axes=rng.choice([1, 1, 2, 3]), pairs=rng.choice(["half", "interleaved"]),
                     norm=rng.random() < 0.6, x=rng.choice(["f16", "f16", "bf16", "f32"]), far=_log(rng, 1, 1 << 20))
            if op == "append":
                c["kt"] = rng.choice(["f16", "f16", "q8_0", "q4_0"])
                c["vt"] = "f16" if c["kt"] == "f16" else rng.choice(["q8_0", "q4_0"])
            else:
                c["out"] = rng.choice(["f16", "f16", "f32"])
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


def _lens(c):
    """Ragged lengths of a batch's sequences, the first one whole."""
    return [max(1, c["n"] - (s * c["n"] * 5) // (8 * max(1, c["S"]))) for s in range(c["S"])]


def _seen(c):
    """Pairs of a token and a key that it sees, over all sequences, of one query head."""
    n, nq = c["n"], c["nq"]
    pairs = 0
    for m in _lens(c) if c["lists"] else [n] * c["S"]:
        t = min(nq, m) if c["lists"] and c["causal"] else nq
        if not c["causal"]:
            pairs += t * (m - c["part"])
        else:                                                 # token i of t sees the keys part .. m - t + i
            first = m - t + 1 - c["part"]                     # keys that the first token sees
            low = max(first, 0)
            high = first + t - 1
            pairs += (high * (high + 1) - low * (low - 1)) // 2 if high >= 0 else 0
    return pairs


def _size(t, D):
    return {"f32": 4 * D, "f16": 2 * D, "bf16": 2 * D, "q8_0": 34 * (D // 32), "q4_0": 18 * (D // 32)}[t]


def work(c):
    H, Hk, D = c["H"], c["Hk"], c["D"]
    if c["op"] == "attn_back":
        T = c["S"] * c["nq"]
        held = sum(_lens(c)) if c["lists"] else c["n"] - c["part"]
        out = c["S"] * c["n"] if c["lists"] else c["n"] - c["part"]
        rows = T * H * (2 * D + 4 * D + 2 * D + 4 + 2 * D)                    # q, o, do, lse read, dq written
        keys = held * Hk * 4 * D + out * Hk * 4 * D                           # k, v read, dk, dv written
        return {"bytes": rows + keys, "flops": 10 * D * H * _seen(c)}
    n, x = c["n"], _size(c["x"], D)
    own_ = n * 4 * c["axes"]
    if c["op"] == "append":
        return {"bytes": own_ + 4 * n + n * (H + 2 * Hk) * x + n * H * 2 * D + n * Hk * (_size(c["kt"], D) + _size(c["vt"], D)), "flops": n * (H + Hk) * D * 10}
    g = _size(c["out"], D)
    if c["op"] == "rope":
        return {"bytes": own_ + n * (H + Hk) * (x + g), "flops": n * (H + Hk) * D * 10}
    return {"bytes": own_ + n * (H + Hk) * (g + x * (2 if c["norm"] else 1)), "flops": n * (H + Hk) * D * 16}


# ------------------------------------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _rows(g, n, heads, D, t):
    """Projections as they come: heads of different size, a few large channels."""
    x = torch.randn((n, heads, D), device="cuda", generator=g)
    x *= torch.rand((heads, 1), device="cuda", generator=g) * 1.5 + 0.5
    x[..., 3::D // 4] *= 4
    return x.to(t)


def prepare(c, seed):
    g = _generator(seed)
    if c["op"] == "attn_back":
        return _prepare_attn(c, g)
    n, H, Hk, D, R, A = c["n"], c["H"], c["Hk"], c["D"], c["R"], c["axes"]
    st = dict(c=c)
    # queries, keys and values as one projection's result
    x = _rows(g, n, H + 2 * Hk, D, TYPES[c["x"]])
    st["q"], st["k"], st["v"] = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    # positions: consecutive ones from `far` on, or a decode step's tokens up to it; further axes walk an image's rows and columns
    t = torch.arange(n, device="cuda")
    if A == 1:
        pos = (c["far"] + t if n > 256 else torch.randint(0, c["far"] + 1, (n,), device="cuda", generator=g)).view(1, n)
    else:
        side = max(1, min(c["far"], 1 << 16))
        pos = torch.stack([t // (side * side), (t // side) % side, t % side][3 - A:])
    st["pos"] = pos.to(torch.int32).contiguous()
    half = R // 2
    st["freq"] = (500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).to(F32)
    # each axis has a section of the pairs; interleaved pairs take turns
    i = torch.arange(half, device="cuda")
    st["axis"] = (i % A if c["pairs"] == "interleaved" else i * A // half).to(torch.int32)
    st["qw"] = st["kw"] = None
    if c["norm"]:
        st["qw"] = 1 + 0.1 * torch.randn(D, device="cuda", generator=g)
        st["kw"] = 1 + 0.1 * torch.randn(D, device="cuda", generator=g)
    if c["op"] == "append":
        rows = n + 37                                       # cache rows, some of them another sequence's
        st["at"] = torch.randperm(rows, device="cuda", generator=g)[:n].to(torch.int32)
        st["kc"] = torch.zeros((rows, Hk * _size(c["kt"], D)), dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros((rows, Hk * _size(c["vt"], D)), dtype=torch.uint8, device="cuda")
        if not c["kt"] == c["vt"] == "f16":
            st["k32"] = torch.empty(rows * Hk * D, dtype=F32, device="cuda")
            st["v32"] = torch.empty(rows * Hk * D, dtype=F32, device="cuda")
    if c["op"] == "rope_back":
        st["dq"] = (torch.randn((n, H, D), device="cuda", generator=g) * 0.02).to(TYPES[c["out"]])
        st["dk"] = (torch.randn((n, Hk, D), device="cuda", generator=g) * 0.02).to(TYPES[c["out"]])
    return st


def _prepare_attn(c, g):
    S, nq, n, H, Hk, D = c["S"], c["nq"], c["n"], c["H"], c["Hk"], c["D"]
    G = H // Hk
    lens = _lens(c) if c["lists"] else None
    rows = sum(lens) if lens else n
    q = (torch.randn((S, nq, H, D), device="cuda", generator=g) * 2).to(F16)
    k = torch.randn((rows, Hk, D), device="cuda", generator=g)
    k += torch.randn((1, Hk, D), device="cuda", generator=g) * 0.5      # what a head's keys have in common
    k = k.to(F16)
    v = torch.randn((rows, Hk, D), device="cuda", generator=g).to(F16)
    do = (torch.randn((S, nq, H, D), device="cuda", generator=g) * 0.05).to(F16)
    st = dict(c=c, q=q, k=k, v=v, do=do, lists=None, pos=None)
    if lens:
        lists = torch.full((S, n), -1, dtype=torch.int32, device="cuda")
        first = 0
        for s, m in enumerate(lens):                          # every second sequence's rows are in no order
            at = torch.randperm(m, device="cuda", generator=g) if s % 2 else torch.arange(m, device="cuda")
            lists[s, :m] = (first + at).to(torch.int32)
            first += m
        st["lists"] = lists
    if c["causal"]:
        t = torch.arange(nq, device="cuda")
        pos = torch.stack([m - min(nq, m) + t if lens else m - nq + t for m in (lens or [n] * S)])
        if lens:                                              # tokens behind a sequence's last one see nothing
            for s, m in enumerate(lens):
                pos[s, min(nq, m):] = -1
        st["pos"] = pos.to(torch.int32).contiguous()
    # the merged output and log-sum-exp over all keys, as the forward pass left them
    o = torch.zeros((S, nq, H, D), dtype=F32, device="cuda")
    lse = torch.full((S, nq, H), -math.inf, dtype=F32, device="cuda")
    for s in range(S):
        r = slice(None) if not lens else lists[s, :lens[s]].long()
        m = n if not lens else lens[s]
        hide = torch.arange(m, device="cuda") > st["pos"][s].view(nq, 1) if c["causal"] else None
        for h in range(H):
            x = (q[s, :, h].float() @ k[r, h // G].float().t()) / math.sqrt(D)
            if hide is not None:
                x.masked_fill_(hide, -math.inf)
            lse[s, :, h] = torch.logsumexp(x, 1)
            o[s, :, h] = torch.exp(x.sub_(lse[s, :, h].unsqueeze(1))).nan_to_num_(0.0) @ v[r, h // G].float()
    st["o"], st["lse"] = o, lse
    return st


# --------------------------------------------------------------------------------------------- the operators

_handle = None


def _own(st):
    """The framework, its handle (kept by the program) and the rotation (kept with its tables)."""
    global _handle
    import split_kv_flash_attn_gb300 as skv
    if _handle is None:
        _handle = skv.Handle(torch.cuda.current_device())
    if "freq" in st and "rope" not in st:
        c = st["c"]
        st["rope"] = skv.Rope(c["D"], st["freq"], axis=st["axis"] if c["axes"] > 1 else None, interleaved=c["pairs"] == "interleaved")
    return skv, _handle


def run(st):
    return {"rope": _rope, "append": _append, "rope_back": _rope_back, "attn_back": _attn_back}[st["c"]["op"]](st)


def _angles(st):
    """cos and sin [n, 1, R/2] of the tokens' angles, which are taken in 64 bits: far positions."""
    a = st["pos"].double()[st["axis"].long()].t() * st["freq"].double()
    return a.cos().float().unsqueeze(1), a.sin().float().unsqueeze(1)


def _pairs(c, x):
    R = c["R"]
    return (x[..., 0:R:2], x[..., 1:R:2]) if c["pairs"] == "interleaved" else (x[..., :R // 2], x[..., R // 2:R])


def _joined(c, a, b, rest):
    turned = torch.stack((a, b), -1).flatten(-2) if c["pairs"] == "interleaved" else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _turn(c, x, cos, sin):
    a, b = _pairs(c, x)
    return _joined(c, a * cos - b * sin, a * sin + b * cos, x[..., c["R"]:])


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def _rope(st):
    if own:
        skv, h = _own(st)
        return skv.rope(h, st["rope"], st["q"], st["k"], st["pos"], q_weight=st["qw"], k_weight=st["kw"], o_dtype=TYPES[st["c"]["out"]])
    c, t = st["c"], TYPES[st["c"]["out"]]
    cos, sin = _angles(st)
    return _turn(c, _normed(st["q"], st["qw"]), cos, sin).to(t), _turn(c, _normed(st["k"], st["kw"]), cos, sin).to(t)


def _held(x, t):
    """fp32 rows [n, Hk, D] as a cache row of this type holds them: the bytes of fp16 rows, or the values of blocks of 32."""
    if t == "f16":
        return x.to(F16)
    most = 127.0 if t == "q8_0" else 7.0
    b = x.view(*x.shape[:2], -1, 32)
    d = (b.abs().amax(-1, keepdim=True) / most).to(F16).float()
    low = -127 if t == "q8_0" else -8
    code = torch.where(d > 0, b / torch.where(d > 0, d, 1.0), 0.0).round().clamp(low, most)
    return (code * d).view_as(x).to(F16)


def _append(st):
    c = st["c"]
    Hk, D = c["Hk"], c["D"]
    quant = "k32" in st
    if own:
        skv, h = _own(st)
        types = {"f16": skv.F16, "q8_0": skv.Q8_0, "q4_0": skv.Q4_0}
        q = skv.rope_append(h, st["rope"], st["q"], st["k"], st["v"], st["pos"], st["at"], st["kc"], st["vc"], q_weight=st["qw"], k_weight=st["kw"],
                            k_type=types[c["kt"]], v_type=types[c["vt"]])
        if not quant:
            return q, st["kc"].view(F16), st["vc"].view(F16)
        # what 8 and 4 bits hold comes back as the values that it stands for
        values = []
        for x, t, out in ((st["kc"], c["kt"], st["k32"]), (st["vc"], c["vt"], st["v32"])):
            (skv.kv_dequant_q8_0 if t == "q8_0" else skv.kv_dequant_q4_0)(h, x, out.numel(), out=out)
            values.append(out.to(F16).view(-1, Hk * D))
        return q, values[0], values[1]
    cos, sin = _angles(st)
    at = st["at"].long()
    q = _turn(c, _normed(st["q"], st["qw"]), cos, sin).to(F16)
    k, v = _held(_turn(c, _normed(st["k"], st["kw"]), cos, sin), c["kt"]), _held(st["v"].float(), c["vt"])
    if quant:
        kc, vc = (torch.zeros((st["kc"].shape[0], Hk * D), dtype=F16, device="cuda") for _ in "kv")
    else:
        kc, vc = st["kc"].view(F16), st["vc"].view(F16)
    kc[at], vc[at] = k.flatten(1), v.flatten(1)
    return q, kc, vc


def _rope_back(st):
    c, x = st["c"], TYPES[st["c"]["x"]]
    if own:
        skv, h = _own(st)
        more = dict(q=st["q"], k=st["k"], q_weight=st["qw"], k_weight=st["kw"]) if c["norm"] else dict(x_dtype=x)
        return skv.rope_backward(h, st["rope"], st["dq"], st["dk"], st["pos"], **more)
    cos, sin = _angles(st)
    dq, dqw = _rows_back(c, st["dq"], st["q"], st["qw"], cos, sin, x)
    dk, dkw = _rows_back(c, st["dk"], st["k"], st["kw"], cos, sin, x)
    return dq, dk, dqw, dkw


def _rows_back(c, dy, x, w, cos, sin, t):
    g = _turn(c, dy.float(), cos, -sin)
    if w is None:
        return g.to(t), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    xr = x * r
    u = g * w
    return (r * (u - xr * (u * xr).mean(-1, keepdim=True))).to(t), (g * xr).sum((0, 1))


def _attn_back(st):
    c = st["c"]
    S, nq, H, D = st["q"].shape
    Hk, part, n = c["Hk"], c["part"], c["n"]
    if own:
        skv, h = _own(st)
        return skv.attn_backward(h, st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], Hk=Hk, kv_begin=part, kv_end=n, kv_rows=st["lists"],
                                 q_pos=st["pos"], g_dtype=F16)
    # [sequence (one, where all share their keys), KV head, query heads x tokens, D]
    shared = st["lists"] is None
    B, T = (1, S * nq) if shared else (S, nq)

    def heads(x):
        return x.float().reshape(B, T, Hk, H // Hk, -1).permute(0, 2, 3, 1, 4).reshape(B, Hk, (H // Hk) * T, -1)

    q, do, o, lse = heads(st["q"]), heads(st["do"]), heads(st["o"]), heads(st["lse"].unsqueeze(-1))
    r = torch.arange(part, n, device="cuda").view(1, -1) if shared else st["lists"].long()
    k, v = (x[r.clamp_min(0)].float().permute(0, 2, 1, 3) for x in (st["k"], st["v"]))
    see = (r >= 0).view(B, 1, 1, -1)
    if c["causal"]:
        see = see & (torch.arange(part, n, device="cuda") <= st["pos"].view(B, 1, T, 1)).repeat(1, 1, H // Hk, 1)
    see = see & (lse > -math.inf)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).sub_(lse)
    p = s.masked_fill_(~see, -math.inf).exp_()
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).masked_fill_(~see, 0.0)
    del p, s
    dq = torch.matmul(ds, k).mul_(1 / math.sqrt(D))
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(1 / math.sqrt(D))
    dq = dq.view(B, Hk, H // Hk, T, D).permute(0, 3, 1, 2, 4).reshape(S, nq, H, D)
    dk, dv = (x.permute(0, 2, 1, 3).to(F16).contiguous() for x in (dk, dv))
    return dq.to(F16), dk[0] if shared else dk, dv[0] if shared else dv


# ------------------------------------------------------------------------------------------ the values in 64 bits

def exact(c, seed):
    st = prepare(c, seed)
    return _exact_attn(st) if c["op"] == "attn_back" else _exact_rows(st)


def _rotated64(st, x):
    """x [n, heads, D] with its pairs as complex numbers, turned."""
    c = st["c"]
    R, half = c["R"], c["R"] // 2
    order = torch.arange(R, device="cuda").view(half, 2) if c["pairs"] == "interleaved" else torch.arange(R, device="cuda").view(2, half).t()
    turn = torch.stack([st["pos"][int(a)].double() * f for a, f in zip(st["axis"].tolist(), st["freq"].double().unbind())], 1)
    z = torch.view_as_complex(x[..., order.reshape(-1)].reshape(*x.shape[:2], half, 2).contiguous())
    z = z * torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
    y = torch.view_as_real(z).flatten(-2)
    back = torch.empty(R, dtype=torch.long, device="cuda")
    back[order.reshape(-1)] = torch.arange(R, device="cuda")
    return torch.cat((y[..., back], x[..., R:]), -1)


def _exact_rows(st):
    c, made = st["c"], []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.double().requires_grad_(c["op"] == "rope_back")
        w = None if w is None else w.double().requires_grad_(c["op"] == "rope_back")
        y = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w
        made.append((x, w, _rotated64(st, y)))
    if c["op"] == "rope":
        return made[0][2], made[1][2]
    if c["op"] == "rope_back":
        rows, weights = [], []
        for (x, w, y), dy in zip(made, (st["dq"], st["dk"])):
            got = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
            rows.append(got[0])
            weights.append(None if w is None else got[1])
        return tuple(rows + weights)
    rows, at, caches = st["kc"].shape[0], st["at"].long(), []
    for x, t in ((made[1][2], c["kt"]), (st["v"].double(), c["vt"])):
        if t != "f16":
            most = 127 if t == "q8_0" else 7
            b = x.reshape(x.shape[0], -1, 32)
            d = (b.abs().max(-1, keepdim=True).values / most).to(F16).double()
            code = (b / d.clamp_min(1e-300)).round().clamp(-127 if t == "q8_0" else -8, most)
            x = torch.where(d > 0, code * d, 0.0)
        full = torch.zeros((rows, c["Hk"] * c["D"]), dtype=torch.float64, device="cuda")
        full[at] = x.reshape(x.shape[0], -1)
        caches.append(full)
    return made[0][2], caches[0], caches[1]


def _exact_attn(st):
    """Autograd through the softmax over all keys, head by head; the partition's keys and the queries that meet them are leaves of their own."""
    c = st["c"]
    S, nq, H, D = st["q"].shape
    Hk, part, n = c["Hk"], c["part"], c["n"]
    G = H // Hk
    shared = st["lists"] is None
    dq = torch.zeros((S, nq, H, D), dtype=torch.float64, device="cuda")
    dk = torch.zeros((1 if shared else S, n - part, Hk, D), dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for s in range(S):
        rows = torch.arange(n, device="cuda") if shared else st["lists"][s][st["lists"][s] >= 0].long()
        m = rows.numel()
        for h in range(H):
            q1 = st["q"][s, :, h].double().requires_grad_()
            q0 = q1.detach()
            k1, v1 = (x[rows[part:], h // G].double().requires_grad_() for x in (st["k"], st["v"]))
            k0, v0 = (x[rows[:part], h // G].double() for x in (st["k"], st["v"]))
            x = torch.cat((q0 @ k0.t(), q1 @ k1.t()), 1) / D ** 0.5
            live = torch.ones(nq, dtype=torch.bool, device="cuda")
            if c["causal"]:
                hide = torch.arange(m, device="cuda") > st["pos"][s].view(nq, 1)
                live = ~hide.all(1)
                x = x.masked_fill(hide & live.view(nq, 1), -math.inf)
            y = torch.softmax(x, 1) @ torch.cat((v0, v1), 0)
            grads = torch.autograd.grad(y, [q1, k1, v1], st["do"][s, :, h].double() * live.view(nq, 1))
            dq[s, :, h] = grads[0]
            dk[0 if shared else s, :m - part, h // G] += grads[1]
            dv[0 if shared else s, :m - part, h // G] += grads[2]
            del x, y, grads
    return (dq, dk[0], dv[0]) if shared else (dq, dk, dv)


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(case, work(case))
