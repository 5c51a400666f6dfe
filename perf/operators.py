"""The 4-bit key/value cache operators as a serving program calls them, and the same in plain torch.

append : a projection's queries, keys and values get their position rotation (and the signed Hadamard rotation of
         keys and queries), keys and values go to the paged 4-bit cache; the appended tokens are read back.
attend : attention of the new queries over the cache (one token, a few, or a prompt's chunk; window and sinks).
step   : append followed by attend, as a model's layer runs them.

Cache layout (one uint8 tensor, pages x kv heads x page (D + 8)): a page of one head holds page x D/2 bytes of key codes,
page x D/2 of value codes, page key words and page value words.  Byte i of a token holds dims 2 i (low half) and 2 i + 1.
A word is the token's fp32 scale with the low 4 bits replaced by the zero point; value = scale (code - zero).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _case(name, kind, B, n, ctx, Hq, Hkv, D, page, dtype, ragged=0, window=0, sinks=0, signs=True, interleaved=False,
          rot=None, causal=True):
    return dict(name=name, kind=kind, B=B, n=n, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, ragged=ragged,
                window=window, sinks=sinks, signs=signs, interleaved=interleaved, rot=D if rot is None else rot,
                causal=causal)


def listed():
    return [
        # one user's next token: launch latency
        _case("append 1 token", "append", 1, 1, 1000, 32, 8, 128, 64, "bf16"),
        # a decode batch's new tokens
        _case("append decode batch", "append", 128, 1, 2048, 32, 8, 128, 64, "fp16", ragged=60),
        # several prompts of different lengths at once
        _case("append prompts", "append", 5, 8192, 8192, 64, 8, 128, 64, "bf16", ragged=50),
        # other head widths, pairs next to each other, part of the head rotated, no Hadamard, odd lengths
        _case("append odd prompts", "append", 3, 1501, 4001, 12, 4, 256, 16, "fp16", ragged=40, signs=False,
              interleaved=True, rot=64),
        # one user's chat
        _case("decode 1 x 8k", "attend", 1, 1, 8191, 32, 8, 128, 64, "bf16"),
        # a busy server
        _case("decode 64 x 8k", "attend", 64, 1, 8192, 64, 8, 128, 64, "bf16", ragged=50),
        # few users, whole books
        _case("decode 4 x 128k", "attend", 4, 1, 131071, 32, 8, 128, 128, "fp16", ragged=20),
        # a model with a sliding window and attention sinks
        _case("decode window", "attend", 32, 1, 32768, 32, 8, 128, 64, "bf16", ragged=30, window=4096, sinks=4),
        # every query head with keys of its own, narrow heads, small pages
        _case("decode mha", "attend", 16, 1, 1030, 32, 32, 64, 16, "fp16", ragged=90),
        # a draft of 5 tokens is appended and verified
        _case("verify a draft", "step", 8, 5, 4000, 32, 8, 128, 32, "bf16", ragged=50),
        # a prompt in chunks: the second chunk over what the first left
        _case("prefill chunk", "attend", 2, 2048, 16384, 32, 8, 128, 64, "bf16"),
        # wide heads, ragged prompts, window and sinks
        _case("prefill window", "attend", 3, 1777, 5003, 16, 4, 256, 64, "fp16", ragged=40, window=1024, sinks=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "attend", "step"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    window, sinks = 0, 0
    if kind != "append" and rng.random() < 0.4:
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 64, 200])
    causal = bool(window or kind != "attend" or rng.random() < 0.85)
    style = rng.random() < 0.3
    rot = rng.choice([0, D // 2, D, D])
    signs = rng.random() < 0.6
    if kind == "append":
        B = _log(rng, 1, 128)
        n = _log(rng, 1, max(1, 24000 // B))
        ctx = n + _log(rng, 1, 4000)
    elif rng.random() < 0.6:
        B = _log(rng, 1, 64)
        n = _log(rng, 1, 9)
        ctx = n + _log(rng, 1, min(100000, 400000 // B))
    else:
        B = _log(rng, 1, 4)
        n = _log(rng, 10, 2500)
        ctx = n + _log(rng, 1, max(1, min(14000, (1 << 30) // (B * Hq * n))))
    return _case("", kind, B, n, ctx, Hq, Hkv, D, page, dtype, ragged=rng.randrange(0, 90), window=window, sinks=sinks,
                 signs=signs, interleaved=style, rot=rot, causal=causal)


def _lens(c):
    """(new tokens, cached tokens with the new ones) of each sequence; the first one has the case's own."""
    n, kv = [], []
    for b in range(c["B"]):
        f = ((b * 37) % 101) * c["ragged"] / 10000.0
        m = max(1, int(c["n"] * (1.0 - f)))
        n.append(m)
        kv.append(max(m, int(c["ctx"] * (1.0 - f)) - (b % 7 if f else 0)))
    return n, kv


def _table(c):
    """(page of each sequence's page slots, -1 behind its last; pages in the pool), the same for every seed."""
    _, kv = _lens(c)
    need = [-(-x // c["page"]) for x in kv]
    pool = sum(need) + 3
    g = torch.Generator().manual_seed(5)
    order = torch.randperm(pool, generator=g).to(torch.int32)
    t = torch.full((c["B"], max(need)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = order[at:at + m]
        at += m
    return t, pool


def prepare(case, seed):
    c = case
    D, Hq, Hkv, page, dt = c["D"], c["Hq"], c["Hkv"], c["page"], DT[c["dtype"]]
    g = torch.Generator("cuda").manual_seed(seed)
    n, kv = _lens(c)
    table, pool = _table(c)
    T = sum(n)
    start = torch.zeros(c["B"] + 1, dtype=torch.int32)
    start[1:] = torch.tensor(n).cumsum(0)
    # a fused projection's output: keys with a few channels of large values
    chan = torch.ones(D, device="cuda")
    chan[torch.randint(0, D, (3,), generator=g, device="cuda")] = 6.0
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")
    qkv[:, Hq:Hq + Hkv] *= chan
    qkv = qkv.to(dt)
    s = dict(case=c, table=table.cuda(), start=start.cuda(), kv=torch.tensor(kv, dtype=torch.int32).cuda(),
             q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], scale=D ** -0.5, rope=None, signs=None)
    if c["rot"]:
        f = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * (
            10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"]))
        s["rope"] = torch.cat([f.cos(), f.sin()], 1).float()
    if c["signs"]:
        s["signs"] = (1 - 2 * torch.randint(0, 2, (D,), generator=g, device="cuda")).to(torch.int8)
    # what earlier tokens left in the cache
    cache = torch.empty(pool, Hkv, page * (D + 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for a in range(0, pool, step):
        m = min(step, pool - a)
        x = torch.randn(m, Hkv, 2, page, D, generator=g, device="cuda")
        if not c["signs"]:
            x[:, :, 0] *= chan
        code, word = _quantize(x)
        cache[a:a + m] = torch.cat([_to_bytes(code).reshape(m, Hkv, -1), word.view(torch.uint8).reshape(m, Hkv, -1)], 2)
    s["cache"] = cache
    return s


# ------------------------------------------------------------- plain form
def _quantize(x):
    """Codes (uint8) and words (int32) of fp32 vectors along the last dimension."""
    lo = x.amin(-1, keepdim=True).clamp_max(0)
    hi = x.amax(-1, keepdim=True).clamp_min(0)
    s = ((hi - lo) * (1.0 / 15.0)).clamp_min(2.0 ** -100)
    bits = torch.bitwise_and(s.view(torch.int32) + 8, -16)
    s = bits.view(torch.float32)
    r = 1.0 / s
    z = (-lo * r).round().clamp(0, 15)
    code = ((x * r).round() + z).clamp(0, 15)
    return code.to(torch.uint8), (bits + z.to(torch.int32)).squeeze(-1)


def _to_bytes(code):
    return code[..., 0::2] + code[..., 1::2] * 16


def _values(codes, words):
    """fp32 values of code bytes (..., D/2) and words (...)."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).float()
    z = (words % 16).float()
    s = torch.bitwise_and(words, -16).view(torch.float32)
    return (c - z[..., None]) * s[..., None]


def _parts(s):
    """The cache as key codes, value codes (pages, heads, page, D/2) and words (pages, heads, 2, page)."""
    c, cache = s["case"], s["cache"]
    P, D = c["page"], c["D"]
    h = P * D // 2
    codes = [cache[..., i * h:(i + 1) * h].unflatten(-1, (P, D // 2)) for i in (0, 1)]
    words = cache.view(torch.int32)[..., P * D // 4:].unflatten(-1, (2, P))
    return codes[0], codes[1], words


def _tokens(s):
    """For each new token: its sequence, index in it, page and slot."""
    T = s["q"].shape[0]
    i = torch.arange(T, device="cuda", dtype=torch.int32)
    b = (torch.searchsorted(s["start"], i, right=True) - 1)
    at = (s["kv"][b] - s["start"][b + 1] + i).long()
    return b, at, s["table"][b, at // s["case"]["page"]].long(), at % s["case"]["page"]


def _rotate(x, at, s):
    """Position rotation and signed Hadamard rotation of (T, H, D), fp32."""
    c, x = s["case"], x.float()
    r = c["rot"]
    if r:
        cs = s["rope"][at][:, None]
        co, si = cs[..., :r // 2], cs[..., r // 2:]
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        y, z = a * co - b * si, b * co + a * si
        y = torch.stack([y, z], -1).flatten(-2) if c["interleaved"] else torch.cat([y, z], -1)
        x = torch.cat([y, x[..., r:]], -1)
    if c["signs"]:
        D = c["D"]
        x = x * s["signs"].float()
        h = 1
        while h < D:
            x = x.unflatten(-1, (D // (2 * h), 2, h))
            x = torch.stack([x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]], -2).flatten(-3)
            h *= 2
        x = x * torch.tensor(D ** -0.5, dtype=torch.float32, device="cuda")
    return x


def _plain_append(s):
    kc, vc, words = _parts(s)
    _, at, page, slot = _tokens(s)
    q = _rotate(s["q"], at, s).to(s["q"].dtype)
    code, word = _quantize(_rotate(s["k"], at, s))
    kc[page, :, slot] = _to_bytes(code)
    words[page, :, 0, slot] = word
    code, word = _quantize(s["v"].float())
    vc[page, :, slot] = _to_bytes(code)
    words[page, :, 1, slot] = word
    return q


def _plain_gather(s):
    kc, vc, words = _parts(s)
    _, _, page, slot = _tokens(s)
    dt = s["q"].dtype
    return (_values(kc[page, :, slot], words[page, :, 0, slot]).to(dt),
            _values(vc[page, :, slot], words[page, :, 1, slot]).to(dt))


def _plain_attend(s, q):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv
    kc, vc, words = _parts(s)
    L = s["table"].shape[1] * c["page"]
    pages = s["table"].clamp_min(0).long()
    # keys and values as (B, Hkv, L, D); new queries padded to the longest sequence's
    k = _values(kc[pages], words[pages][:, :, :, 0]).transpose(1, 2).reshape(B, Hkv, L, D)
    v = _values(vc[pages], words[pages][:, :, :, 1]).transpose(1, 2).reshape(B, Hkv, L, D)
    n = s["start"][1:] - s["start"][:-1]
    N = c["n"]
    b, at, _, _ = _tokens(s)
    i = (at - (s["kv"] - n)[b]).long()
    qp = torch.zeros(B, N, Hq, D, device="cuda")
    qp[b, i] = q.float()
    qp = qp.unflatten(2, (Hkv, g)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * g, D)
    x = (qp @ k.transpose(-1, -2)).mul_(s["scale"])
    j = torch.arange(L, device="cuda")
    p = ((s["kv"] - n)[:, None] + torch.arange(N, device="cuda")).repeat_interleave(g, 1)[:, :, None]
    seen = j < s["kv"][:, None, None]
    if c["causal"]:
        seen = seen & (j <= p)
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    x.masked_fill_(~seen[:, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x @ v).div_(l).unflatten(2, (N, g)).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    return o[b, i].to(q.dtype)


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["kind"] == "append":
        q = _plain_append(s)
        return (q, *_plain_gather(s))
    if c["kind"] == "step":
        q = _plain_append(s)
        return q, _plain_attend(s, q)
    return _plain_attend(s, s["q"])


def _run_own(s, c):
    from post_quantization_02_b200 import kv4

    batch = (s["table"], s["start"], s["kv"])
    q = s["q"]
    if c["kind"] != "attend":
        q = kv4.append(s["q"], s["k"], s["v"], s["cache"], *batch, rope=s["rope"], interleaved=c["interleaved"],
                       signs=s["signs"])
        if c["kind"] == "append":
            return (q, *kv4.gather(s["cache"], *batch, tokens=q.shape[0], head_dim=c["D"], dtype=q.dtype))
    o = kv4.attend(q, s["cache"], *batch, scale=s["scale"], causal=c["causal"], window=c["window"], sinks=c["sinks"])
    return (q, o) if c["kind"] == "step" else o


# -------------------------------------------------------------------- work
def _visible(c):
    """(pairs of query and visible key, keys that some query sees), over all sequences, for one head."""
    pairs = keys = 0
    for n, kv in zip(*_lens(c)):
        w, k0 = c["window"], c["sinks"]
        if not c["causal"]:
            pairs, keys = pairs + n * kv, keys + kv
            continue
        first = kv - n
        if not w:
            pairs += n * first + n * (n + 1) // 2
            keys += kv
            continue
        for p in range(first, kv):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(k0, lo)
        lo = max(0, first - w + 1)
        keys += kv - lo + min(k0, lo)
    return pairs, keys


def work(case):
    c = case
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    T = sum(_lens(c)[0])
    cached, wide = Hkv * (D + 8), Hkv * 2 * D * 2
    put = T * (wide + cached + 2 * Hq * D * 2) + (T * c["rot"] * 4 if c["rot"] else 0)
    if c["kind"] == "append":
        # read q, k, v and the angles; write q and the cache; the read-back reads the cache and writes values
        lg = int(math.log2(D)) if c["signs"] else 0
        per = (Hq + Hkv) * (3 * c["rot"] + D * lg) + 2 * Hkv * D * 6 + 2 * Hkv * D * 2
        return {"bytes": put + T * (cached + wide), "flops": T * per}
    pairs, keys = _visible(c)
    b = keys * cached + 2 * T * Hq * D * 2
    if c["kind"] == "step":
        b += put
    return {"bytes": b, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------- exact
def _grid64(w):
    lo = torch.minimum(w.min(-1).values, torch.zeros((), dtype=w.dtype, device=w.device))
    hi = torch.maximum(w.max(-1).values, torch.zeros((), dtype=w.dtype, device=w.device))
    # the stored scale has 20 bits: the low 4 of an fp32 number's 24 hold the zero point
    m, e = torch.frexp(((hi - lo) / 15).clamp_min(2.0 ** -100))
    s = torch.ldexp(torch.floor(m * 2 ** 20 + 0.5), e - 20)
    z = torch.clamp(torch.round(-lo / s), 0, 15)
    q = torch.clamp(torch.round(w / s[..., None]) + z[..., None], 0, 15)
    return s[..., None] * (q - z[..., None])


def _turn64(x, pos, s):
    c = s["case"]
    x = x.double().clone()
    r = c["rot"]
    if r:
        t = s["rope"].double()[pos][:, None, :]
        h = r // 2
        even = torch.arange(0, r, 2, device=x.device) if c["interleaved"] else torch.arange(h, device=x.device)
        odd = even + (1 if c["interleaved"] else h)
        a, b = x[..., even], x[..., odd]
        x[..., even] = a * t[..., :h] - b * t[..., h:]
        x[..., odd] = a * t[..., h:] + b * t[..., :h]
    if c["signs"]:
        H = torch.ones(1, 1, dtype=torch.float64, device=x.device)
        while H.shape[0] < c["D"]:
            H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
        x = (x * s["signs"].double()) @ H / math.sqrt(c["D"])
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    D, Hkv, P = c["D"], c["Hkv"], c["page"]
    g = c["Hq"] // Hkv
    half = P * D // 2
    rows = {"q": [], "k": [], "v": [], "o": []}
    start = s["start"].tolist()
    for b, (n, kv) in enumerate(zip(*_lens(c))):
        new = slice(start[b], start[b] + n)
        pos = torch.arange(kv - n, kv, device="cuda")
        if c["kind"] == "attend":
            q = s["q"][new].double()
        else:
            q = _turn64(s["q"][new], pos, s)
            kn, vn = _grid64(_turn64(s["k"][new], pos, s)), _grid64(s["v"][new].double())
            if c["kind"] == "append":
                rows["k"].append(kn)
                rows["v"].append(vn)
            else:
                # attention sees the queries as they are handed on: in their own type
                rows["q"].append(q)
                q = q.to(DT[c["dtype"]]).double()
        if c["kind"] == "append":
            rows["q"].append(q)
            continue
        pages = s["table"][b, :-(-kv // P)].long()
        raw = s["cache"][pages]
        kvv = []
        for i in (0, 1):
            by = raw[..., i * half:(i + 1) * half].reshape(-1, Hkv, P, D // 2)
            code = torch.zeros(by.shape[:-1] + (D,), dtype=torch.float64, device="cuda")
            code[..., 0::2] = (by & 15).double()
            code[..., 1::2] = (by >> 4).double()
            w = raw[..., 2 * half + 4 * P * i:2 * half + 4 * P * (i + 1)].contiguous().view(torch.int32)
            val = (code - (w & 15).double()[..., None]) * (w & ~15).view(torch.float32).double()[..., None]
            kvv.append(val.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :kv])
        k, v = kvv
        if c["kind"] == "step":
            k[:, kv - n:], v[:, kv - n:] = kn.transpose(0, 1), vn.transpose(0, 1)
        j = torch.arange(kv, device="cuda")
        out = []
        for a in range(0, n, 256):
            p = pos[a:a + 256, None]
            ok = (j <= p) if c["causal"] else (j >= 0).expand(p.shape[0], kv)
            if c["window"]:
                ok = ok & ((p - j < c["window"]) | (j < c["sinks"]))
            qq = q[a:a + 256].reshape(-1, Hkv, g, D)
            x = torch.einsum("nhgd,hjd->hgnj", qq, k) * s["scale"]
            x = torch.softmax(x.masked_fill(~ok, -math.inf), -1)
            out.append(torch.einsum("hgnj,hjd->nhgd", x, v).reshape(-1, c["Hq"], D))
        rows["o"].append(torch.cat(out))
    cat = {k: torch.cat(v) for k, v in rows.items() if v}
    if c["kind"] == "append":
        return cat["q"], cat["k"], cat["v"]
    if c["kind"] == "step":
        return cat["q"], cat["o"]
    return cat["o"]
