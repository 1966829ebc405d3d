"""What is measured of the operators over a paged cache of keys and values.

Four operators share one description of a batch.  A cache holds pages of S rows
for each of Hkv heads, [pages, Hkv, S, D] in bf16, or in 4 bits: a byte j of a
row holds the codes of channels j (low half) and j + D/2 (high half), and each
row has a scale and a smallest value (bf16 both), a code c standing for
min + scale * c.  page_table[b] names the pages of sequence b in order;
seq_lens[b] counts its tokens, the new ones included; q_starts packs the new
tokens of all sequences into one axis.

- append: rotates the new keys (and queries) to their positions and stores keys
  and values in their places;
- read: the rows of the batch's tokens back in bf16 (after an append into a
  4-bit cache, whose contents are values only through it);
- attn: each new token's attention over its sequence up to itself, from bf16
  or 4-bit pages.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one new token of each of 4 conversations: what a small server does per layer and step
        dict(name="append 4 tokens", op="append", bits=16, B=4, new_lo=1, new_hi=1, len_lo=900, len_hi=1100, H=32,
             Hkv=8, D=128, S=16, scale=1.0),
        # four prompts of uneven length, about the long workload's 32768 tokens in all, at interpolated positions
        dict(name="append prompts", op="append", bits=16, B=4, new_lo=3500, new_hi=12900, len_lo=0, len_hi=0, H=32,
             Hkv=8, D=128, S=64, scale=0.25),
        # single tokens into a 4-bit cache of small heads, and the rows looked at again
        dict(name="append read 4-bit 7 tokens", op="append_read", bits=4, B=7, new_lo=1, new_hi=1, len_lo=100,
             len_hi=900, H=16, Hkv=8, D=64, S=32, scale=1.0),
        # three prompts into a 4-bit cache, read back as the dense forward takes them
        dict(name="append read 4-bit prompts", op="append_read", bits=4, B=3, new_lo=2731, new_hi=9001, len_lo=0,
             len_hi=0, H=32, Hkv=8, D=128, S=64, scale=1.0),
        # the smallest step: one token of one short conversation, a key head for each query head
        dict(name="decode 1 x 513", op="attn", bits=16, B=1, new_lo=1, new_hi=1, len_lo=513, len_hi=513, H=32, Hkv=32,
             D=128, S=16, scale=1.0),
        # one long document (the long workload's length), grouped heads
        dict(name="decode 1 x 32768", op="attn", bits=16, B=1, new_lo=1, new_hi=1, len_lo=32768, len_hi=32768, H=32,
             Hkv=8, D=128, S=64, scale=1.0),
        # a busy server: 64 conversations of very different lengths
        dict(name="decode 64 ragged", op="attn", bits=16, B=64, new_lo=1, new_hi=1, len_lo=17, len_hi=8192, H=32,
             Hkv=8, D=128, S=16, scale=1.0),
        # a chunk of a long prompt over what came before it: compute bound, the largest
        dict(name="chunk 2048 over 16384", op="attn", bits=16, B=1, new_lo=2048, new_hi=2048, len_lo=16384,
             len_hi=16384, H=32, Hkv=8, D=128, S=64, scale=1.0),
        # a very long document held in 4 bits
        dict(name="decode 4-bit 1 x 131072", op="attn", bits=4, B=1, new_lo=1, new_hi=1, len_lo=131072,
             len_hi=131072, H=32, Hkv=8, D=128, S=64, scale=1.0),
        # many conversations in 4 bits, a key head for each query head
        dict(name="decode 4-bit 48 ragged", op="attn", bits=4, B=48, new_lo=1, new_hi=1, len_lo=33, len_hi=4096, H=32,
             Hkv=32, D=128, S=32, scale=1.0),
        # a few guessed tokens of each conversation checked at once
        dict(name="decode 4-bit 16 x 5 new", op="attn", bits=4, B=16, new_lo=5, new_hi=5, len_lo=300, len_hi=6001,
             H=16, Hkv=2, D=64, S=16, scale=1.0),
        # uneven prompt chunks over 4-bit pages
        dict(name="chunk 4-bit ragged", op="attn", bits=4, B=3, new_lo=260, new_hi=1000, len_lo=3001, len_hi=12000,
             H=32, Hkv=8, D=128, S=128, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.6e15)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["append", "append_read", "attn", "attn", "attn", "attn"])
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8, 8, 32])
        g = rng.choice([1, 1, 2, 3, 4, 7, 8, 16]) if Hkv <= 4 else rng.choice([1, 2, 4, 8] if Hkv == 8 else [1, 2])
        c = dict(op=op, bits=rng.choice([16, 4]) if op != "append_read" else 4, D=D, H=Hkv * g, Hkv=Hkv,
                 S=rng.choice([16, 32, 64, 128]), scale=rng.choice([1.0, 1.0, 0.25]))
        if op == "append":
            c["bits"] = 16
        if rng.random() < (0.5 if op != "attn" else 0.7):  # a step: one or a few new tokens of each sequence
            c["B"] = _log(rng, 1, 96)
            c["new_lo"] = c["new_hi"] = rng.choice([1, 1, 1, 2, 4, 5])
            hi = _log(rng, 20, 131072 if c["bits"] == 4 else 65536)
            c["len_lo"], c["len_hi"] = rng.choice([(hi, hi), (max(1, hi // 64), hi), (max(1, hi // 3), hi)])
            if op != "attn":  # a step's append does not depend on the length of the past
                c["len_hi"] = min(c["len_hi"], 2000)
                c["len_lo"] = min(c["len_lo"], c["len_hi"])
        else:  # prompts, or chunks of them
            c["B"] = _log(rng, 1, 6)
            c["new_hi"] = _log(rng, 20, 8000 if op != "attn" else 2000)
            c["new_lo"] = rng.randint(max(1, c["new_hi"] // 3), c["new_hi"])
            past = rng.choice([0, _log(rng, 1, 16000)]) if op == "attn" else 0
            c["len_lo"], c["len_hi"] = rng.randint(past // 2, past), past
        # the plain form holds every score and every key in 32 bits, padded to the longest sequence
        lens, news = _lens(c)
        if max(lens) * c["B"] * (c["H"] * max(news) + 3 * Hkv * D) * 4 > 30e9 or _cost(c) > most:
            continue
        return c


def _lens(c):
    """Tokens of each sequence (new ones included) and its new tokens: the case's alone, spread over its ranges."""
    lens, news = [], []
    for b in range(c["B"]):
        u = ((b + 1) * GOLDEN) % 1.0
        w = ((b + 1) * GOLDEN * GOLDEN + 0.31) % 1.0
        n = c["new_lo"] + int(round(u * (c["new_hi"] - c["new_lo"])))
        news.append(n)
        lens.append(max(n, c["len_lo"] + int(round(w * (c["len_hi"] - c["len_lo"])))))
    return lens, news


def work(c):
    lens, news = _lens(c)
    H, Hkv, D, T = c["H"], c["Hkv"], c["D"], sum(news)
    row = 2 * D if c["bits"] == 16 else D // 2 + 4  # bytes of a stored row of one head
    if c["op"] == "attn":
        pairs = sum(n * l - n * (n - 1) // 2 for l, n in zip(lens, news))
        return {"bytes": sum(lens) * 2 * Hkv * row + 2 * T * H * D * 2, "flops": 4.0 * H * D * pairs}
    b = T * (2 * H * D * 2 + 2 * Hkv * D * 2 + 2 * Hkv * row)
    f = 3.0 * T * (H + Hkv) * D
    if c["op"] == "append_read":
        b += T * 2 * Hkv * (row + 2 * D)
        f += 6.0 * T * Hkv * D
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- inputs


def _pack(x):
    """Rows [..., D] (bf16) in 4 bits: codes [..., D/2] uint8, (scale, min) [..., 2] bf16."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16().float()
    c = torch.where(s > 0, torch.round((x - lo) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15).to(torch.uint8)
    half = x.shape[-1] // 2
    return c[..., :half] | (c[..., half:] << 4), torch.cat([s, lo], -1).bfloat16()


def _unpack(codes, scale):
    """The values that 4-bit rows stand for, in 32 bits."""
    c = torch.cat([codes & 15, codes >> 4], -1).float()
    return scale[..., 1:].float() + scale[..., :1].float() * c


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, news = _lens(c)
    B, H, Hkv, D, S, T = c["B"], c["H"], c["Hkv"], c["D"], c["S"], sum(news)
    need = [-(-l // S) for l in lens]
    wide = max(need) + 1
    pages = sum(need) + 3
    # pages in the order in which a busy allocator hands them out: none; entries behind a sequence name no page
    ids = torch.randperm(pages, generator=gen, device=dev)[:sum(need)].to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device=dev)
    n_of = torch.tensor(need, device=dev)
    table[torch.arange(wide, device=dev) < n_of[:, None]] = ids
    starts = torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32)
    st = dict(case=c, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), starts=starts, T=T,
              max_new=max(news), max_len=max(lens), base=10000.0, scale=c["scale"])
    # keys with a few strong channels, as rotated keys have, and values around zero; one row in twenty has twice the key
    amp = 1.0 + 2.0 * (torch.rand(Hkv, 1, D, generator=gen, device=dev) < 0.03).float()
    shape = (pages, Hkv, S, D)
    k = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    k *= amp.bfloat16()
    k *= 1 + (torch.rand(pages, 1, S, 1, generator=gen, device=dev) < 0.05).bfloat16()
    v = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    if c["bits"] == 16:
        st.update(k=k, v=v, ks=None, vs=None)
    else:
        (kc, ks), (vc, vs) = _pack(k), _pack(v)
        st.update(k=kc, v=vc, ks=ks, vs=vs)
    del k, v
    # new tokens as the projection leaves them: q, k and v of a token side by side in one row
    qkv = torch.randn(T, (H + 2 * Hkv) * D, generator=gen, device=dev, dtype=torch.bfloat16)
    st["q"] = qkv[:, : H * D].unflatten(1, (H, D))
    st["nk"] = qkv[:, H * D : (H + Hkv) * D].unflatten(1, (Hkv, D))
    st["nv"] = qkv[:, (H + Hkv) * D :].unflatten(1, (Hkv, D))
    st["out"] = torch.empty(T, H, D, device=dev, dtype=torch.bfloat16)
    if own:  # the handles and the workspace that a serving program keeps over its steps
        import shifted_sparse_attention_b200 as s2

        st["cache"] = s2.KVCache(st["k"], st["v"], st["ks"], st["vs"])
        st["batch"] = s2.CacheBatch(table, st["lens"], starts, T, max_new=st["max_new"], max_len=st["max_len"])
        st["ws"] = s2.cache_attention_workspace(st["cache"], st["batch"], H) if c["op"] == "attn" else None
        st["rows"] = (torch.empty(T, Hkv, D, device=dev, dtype=torch.bfloat16),
                      torch.empty(T, Hkv, D, device=dev, dtype=torch.bfloat16))
    return st


# ---------------------------------------------------------------- the operators


def _places(st):
    """Sequence, place in it, page and slot of each new token."""
    t = torch.arange(st["T"], device=st["table"].device)
    b = torch.searchsorted(st["starts"].long(), t, right=True) - 1
    p = st["lens"].long()[b] - st["starts"].long()[b + 1] + t
    S = st["case"]["S"]
    return b, p, st["table"].long()[b, p // S], p % S


def _rotate(x, p, base, scale):
    """Rotation by angles formed in 64 bits, in 32 bits, rounded once."""
    half = x.shape[-1] // 2
    j = torch.arange(half, device=x.device, dtype=torch.float64)
    a = p.double()[:, None] * scale * base ** (-2.0 * j / x.shape[-1])
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    lo, hi = x[..., :half].float(), x[..., half:].float()
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).bfloat16()


def _append(st):
    b, p, page, slot = _places(st)
    k, v = _rotate(st["nk"], p, st["base"], st["scale"]), st["nv"]
    q = _rotate(st["q"], p, st["base"], st["scale"])
    if st["ks"] is None:
        st["k"][page, :, slot] = k
        st["v"][page, :, slot] = v
    else:
        for x, codes, scale in ((k, st["k"], st["ks"]), (v, st["v"], st["vs"])):
            c, s = _pack(x)
            codes[page, :, slot] = c
            scale[page, :, slot] = s
    return q, page, slot


def _attn(st):
    c, B, Hkv, D = st["case"], st["case"]["B"], st["case"]["Hkv"], st["case"]["D"]
    g, table = c["H"] // Hkv, st["table"].long().clamp(min=0)
    k, v = st["k"][table], st["v"][table]  # [B, pages, Hkv, S, D]
    if st["ks"] is not None:
        k, v = _unpack(k, st["ks"][table]), _unpack(v, st["vs"][table])
    k, v = (x.float().transpose(1, 2).flatten(2, 3) for x in (k, v))
    n, starts, lens = st["max_new"], st["starts"].long(), st["lens"].long()
    i = torch.arange(n, device=table.device)
    new = starts.diff()
    t = (starts[:-1, None] + i).clamp(max=st["T"] - 1)  # [B, n]; sequences with fewer new tokens repeat others' rows
    q = st["q"][t].float().reshape(B, n, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * g, D)
    s = q @ k.transpose(2, 3)
    s *= 1.0 / math.sqrt(D)
    place = (lens - new)[:, None] + i
    seen = torch.arange(k.shape[2], device=table.device) <= place[..., None]  # [B, n, L]
    s = s.view(B, Hkv, n, g, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.reshape(B, Hkv, n * g, -1) @ v).view(B, Hkv, n, g, D) / total
    mine = i < new[:, None]  # [B, n]: in order of b and i, the packed order of the tokens
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, c["H"], D)[mine].bfloat16()


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import shifted_sparse_attention_b200 as s2

        if op == "attn":
            return s2.cache_attention(st["cache"], st["batch"], st["q"], out=st["out"], workspace=st["ws"])
        q = s2.cache_append(st["cache"], st["batch"], st["nk"], st["nv"], st["q"], base=st["base"], scale=st["scale"],
                            out=st["out"])
        if op == "append":
            return q, st["k"], st["v"]
        return (q, *s2.cache_read(st["cache"], st["batch"], out=st["rows"]))
    if op == "attn":
        return _attn(st)
    q, page, slot = _append(st)
    if op == "append":
        return q, st["k"], st["v"]
    return (q, _unpack(st["k"][page, :, slot], st["ks"][page, :, slot]).bfloat16(),
            _unpack(st["v"][page, :, slot], st["vs"][page, :, slot]).bfloat16())


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """Sequence by sequence and head by head, from the definitions above."""
    st = prepare(case, seed)
    c, dev = case, st["table"].device
    lens, news = _lens(c)
    H, Hkv, D, S = c["H"], c["Hkv"], c["D"], c["S"]
    half, g = D // 2, H // Hkv

    def values(codes, pair):
        x = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device=dev)
        x[..., :half] = codes.to(torch.int64).remainder(16).double()
        x[..., half:] = torch.div(codes.to(torch.int64), 16, rounding_mode="floor").double()
        return x * pair[..., 0:1].double() + pair[..., 1:2].double()

    if c["op"] == "attn":
        if work(c)["flops"] > 2e12:
            return None
        out, at = torch.empty(st["T"], H, D, dtype=torch.float64, device=dev), 0
        for b, (l, n) in enumerate(zip(lens, news)):
            ids = st["table"][b, : -(-l // S)].long()
            pos = torch.arange(l - n, l, device=dev)
            for h in range(Hkv):
                k, v = st["k"][ids, h].reshape(len(ids) * S, -1)[:l], st["v"][ids, h].reshape(len(ids) * S, -1)[:l]
                if st["ks"] is None:
                    k, v = k.double(), v.double()
                else:
                    k = values(k, st["ks"][ids, h].reshape(-1, 2)[:l])
                    v = values(v, st["vs"][ids, h].reshape(-1, 2)[:l])
                for y in range(h * g, (h + 1) * g):
                    z = st["q"][at : at + n, y].double() @ k.T / math.sqrt(D)
                    if n > 1:
                        z[torch.arange(l, device=dev)[None, :] > pos[:, None]] = -math.inf
                    out[at : at + n, y] = torch.softmax(z, -1) @ v
            at += n
        return out

    where = torch.cat([torch.arange(l - n, l, device=dev) for l, n in zip(lens, news)]).double()
    freq = torch.tensor([10000.0 ** (-j / half) for j in range(half)], dtype=torch.float64, device=dev)
    angle = (where * c["scale"])[:, None, None] * freq
    turn = torch.polar(torch.ones_like(angle), angle)

    def turned(x):
        z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turn
        return torch.cat([z.real, z.imag], -1)

    q, k, v = turned(st["q"]), turned(st["nk"]), st["nv"].double()
    if c["op"] == "append_read":
        rows = []
        for x in (k, v):
            x = x.bfloat16().double()  # a row is packed as bf16 holds it
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            s = ((hi - lo) / 15).bfloat16().double()
            rows.append(lo + s * ((x - lo) / s).round().clamp(0, 15))
        return (q, *rows)
    kept, at = [st["k"].double(), st["v"].double()], 0
    for b, (l, n) in enumerate(zip(lens, news)):
        p = torch.arange(l - n, l, device=dev)
        page = st["table"][b].long()[p // S]
        for store, x in zip(kept, (k, v)):
            store[page, :, p % S] = x[at : at + n]
        at += n
    return (q, *kept)
