"""The 4-bit key/value cache on the GPU against its host oracle (oracle/kv4.py).

Append is compared bit for bit (codes, words, and the rotated queries, which are
one rounding of fp32 values the oracle has exactly).  Attention is compared
element by element with a bound taken from the kernel's roundings: with p the
exact probabilities, V the cached values and o the exact output,

  |err| <= eps/2 |o|                       the output's rounding
         + (2^-11 + 2 Ex) sum_j p_j |V_j|  probabilities rounded to fp16, scores off by Ex
         + Ea sum_j p_j s_j 30             fp32 sums of codes and of zero points

Ex: scores are sums of head_dim fp16 x 4-bit products in fp32: head_dim roundings
(counted at 2^-23, a truncating sum) of at most scale sum_d |q_d| s_j 15, twice
(codes, zero point).  Ea: one rounding of 2^-23 per 16 keys and 64 for joins.

Many rows per key and bf16 queries: keys and values themselves are rounded to fp16.
A key's dim is off by 2^-11 |k_jd|, and by 2^-25 of a step's largest scale where it
is a subnormal: Ex gets scale sum_d |q_d| (2^-11 |k_jd| + 2^-24 15 max s).  A value is
the rounded product of its codes and its rounded scale: two more 2^-11 sum_j p_j |V_j|.
"""

import numpy as np
import pytest
import torch

from gpu_helpers import t
from oracle import kv4 as ok
from post_quantization_02_b200 import abi, kv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def f64(x):
    return x.detach().to(torch.float64).cpu().numpy()


class Setup:
    """A pool of pages full of bytes that read as NaN, and a batch in it."""

    def __init__(self, dev, r, new, kv, heads, D, P, spare=2, extra=0):
        self.dev, self.P, self.D, self.heads = dev, P, D, heads
        self.new, self.kv = list(new), list(kv)
        need = [-(-x // P) for x in kv]
        self.pages = sum(need) + spare
        self.cache = kv4.make_cache(self.pages, P, heads, D, dev)
        self.cache.fill_(255)
        perm = r.permutation(self.pages)
        width = max(need + [0]) + extra
        bt = np.full((len(kv), width), -7, dtype=np.int32)
        at = 0
        for b, m in enumerate(need):
            bt[b, :m] = perm[at:at + m]
            at += m
        self.bt = bt
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.args = (t(bt, dev), t(self.start, dev), i32(self.kv, dev))
        self.T = int(self.start[-1])

    def fill(self, r, lo=0):
        """Tokens lo .. kv of every sequence as an append of random vectors leaves them."""
        raw = self.cache.cpu().numpy()
        for b, L in enumerate(self.kv):
            for j in range(lo, L):
                blk = raw[self.bt[b, j // self.P]]
                x = r.standard_normal((self.heads, 2, self.D)) * np.exp(r.normal(0, 0.5, (self.heads, 2, 1)))
                c, s, z = ok.quantize(x)
                w = ok.words(s, z)
                for h in range(self.heads):
                    for i in (0, 1):
                        ok.put(blk[h], self.P, self.D, j % self.P, c[h, i], w[h, i], i)
        self.cache.copy_(torch.from_numpy(raw))

    def fill_fast(self, dev_gen):
        """The same with random codes and scales, on the device (long sequences)."""
        P, D = self.P, self.D
        n = self.pages * self.heads
        codes = torch.randint(0, 256, (n, P * D), generator=dev_gen, device=self.dev, dtype=torch.int32).to(torch.uint8)
        s = torch.rand(n, 2 * P, generator=dev_gen, device=self.dev) * 0.3 + 0.05
        z = torch.randint(5, 11, (n, 2 * P), generator=dev_gen, device=self.dev, dtype=torch.int32)
        w = (s.view(torch.int32) & -16) | z
        self.cache.view(n, -1).copy_(torch.cat([codes, w.view(torch.uint8).view(n, -1)], 1))

    def host(self, b):
        """(keys, values, key scales, value scales) of sequence b, fp64, (heads, L, ...)."""
        L, P = self.kv[b], self.P
        m = -(-L // P)
        raw = self.cache[t(self.bt[b, :m].astype(np.int64), self.dev)].cpu().numpy()
        kc, vc, kw, vw = ok.split_block(raw, P, self.D)
        flat = lambda x: np.moveaxis(x, 1, 0).reshape((self.heads, m * P) + x.shape[3:])[:, :L]  # noqa: E731
        k, v = ok.values(flat(kc), flat(kw)), ok.values(flat(vc), flat(vw))
        sc = lambda w: (flat(w) & np.uint32(0xFFFFFFF0)).view(np.float32).astype(np.float64)  # noqa: E731
        return k, v, sc(kw), sc(vw)


def check_attention(st, q, out, scale, causal=True, window=0, sinks=0, lse=None, rows=None, seqs=None):
    dt = q.dtype
    eps = torch.finfo(dt).eps
    qh, oh = f64(q), f64(out)
    g = q.shape[1] // st.heads
    rounded = dt == torch.bfloat16 and st.start[-1] * g > (40 if st.D == 256 else 64) * len(st.kv)
    for b in range(len(st.kv)) if seqs is None else seqs:
        if st.new[b] == 0:
            continue
        k, v, ks, vs = st.host(b)
        L = st.kv[b]
        todo = range(st.new[b]) if rows is None else sorted({min(x, st.new[b] - 1) for x in rows})
        for i in todo:
            p = L - st.new[b] + i
            mask = ok.visible(p, L, causal, window, sinks)
            row = st.start[b] + i
            for h in range(q.shape[1]):
                kh = h // g
                o, ls, pr = ok.attend(qh[row, h], k[kh], v[kh], scale, mask)
                got = oh[row, h]
                if not mask.any():
                    assert not got.any()
                    assert lse is None or lse[row, h].item() == -np.inf
                    continue
                pr, vh = pr[mask], v[kh][mask]
                ex = 2 * st.D * 2.0 ** -23 * scale * np.abs(qh[row, h]).sum() * 15 * ks[kh][mask].max()
                if rounded:
                    qa = np.abs(qh[row, h])
                    ex += scale * (2.0 ** -11 * (np.abs(k[kh][mask]) @ qa).max()
                                   + 2.0 ** -24 * 15 * qa.sum() * ks[kh][mask].max())
                ea = 2.0 ** -23 * (mask.sum() / 16 + 64)
                tol = (eps / 2 * np.abs(o) + ((3 if rounded else 1) * 2.0 ** -11 + 2 * ex) * (pr @ np.abs(vh))
                       + ea * 30 * (pr @ vs[kh][mask]) + torch.finfo(dt).tiny)
                bad = np.abs(got - o) > tol
                assert not bad.any(), (b, i, h, np.abs(got - o)[bad][:4], tol[bad][:4])
                if lse is not None:
                    assert abs(lse[row, h].item() - ls) <= ex + 2.0 ** -20 * (1 + abs(ls))


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("D,P,heads,Hq,dtype,rot,inter,signs,new,kv", [
    (128, 16, 2, 4, "bf16", 128, False, True, [1, 5, 0, 3], [1, 40, 0, 3]),
    (64, 32, 3, 3, "fp16", 64, False, True, [2, 33], [2, 64]),
    (256, 64, 1, 5, "bf16", 256, False, False, [4], [130]),
    (128, 64, 2, 2, "fp16", 32, False, False, [3, 1], [7, 64]),
    (128, 128, 1, 4, "bf16", 48, True, True, [3], [300]),
    (64, 16, 2, 2, "bf16", 0, False, True, [17], [17]),
    (256, 256, 2, 4, "fp16", 256, True, True, [2, 2], [257, 2]),
    (128, 16, 1, 0, "bf16", 128, True, False, [6], [21]),
])
def test_append_bit_exact(cuda, D, P, heads, Hq, dtype, rot, inter, signs, new, kv):
    r = np.random.default_rng(D + P + rot)
    st = Setup(cuda, r, new, kv, heads, D, P, extra=1)
    dt = DT[dtype]
    T = st.T + 2                                   # two rows of padding at the end
    x = torch.from_numpy(r.standard_normal((T, Hq + 2 * heads, D)) * np.exp(r.normal(0, 1, (1, 1, D)))).to(cuda, dt)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + heads], x[:, Hq + heads:]
    rows = max(kv) + 1
    tab = r.standard_normal((rows, rot)).astype(np.float32) if rot else None
    sg = (1 - 2 * r.integers(0, 2, D)).astype(np.int8) if signs else None
    before = st.cache.cpu().numpy()
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    q_out = torch.full((T, Hq, D), 7.0, dtype=dt, device=cuda) if Hq else None
    kv4.append(q if Hq else None, k, v, st.cache, *st.args, rope=None if tab is None else t(tab, cuda),
               interleaved=inter, signs=None if sg is None else t(sg, cuda), q_out=q_out, info=info)
    assert info.item() == 0
    xh = x.float().cpu().numpy()
    want = before.copy()
    for b in range(len(kv)):
        for i in range(new[b]):
            at, row = kv[b] - new[b] + i, st.start[b] + i
            tr = tab[at] if rot else None
            kr = ok.rotate(xh[row, Hq:Hq + heads], tr, rot, inter, sg)
            for isv, vec in ((0, kr), (1, xh[row, Hq + heads:])):
                c, s, z = ok.quantize(vec)
                w = ok.words(s, z)
                for h in range(heads):
                    ok.put(want[st.bt[b, at // P], h], P, D, at % P, c[h], w[h], isv)
            if Hq:
                qr = torch.from_numpy(ok.rotate(xh[row, :Hq], tr, rot, inter, sg)).to(dt)
                assert torch.equal(q_out[row].cpu(), qr)
    assert np.array_equal(st.cache.cpu().numpy(), want)
    if Hq:
        assert (q_out[st.T:] == 7).all()           # padding rows are left as they were


@pytest.mark.parametrize("off,st_t,st_h", [(1, 0, 0), (0, 3, 0), (0, 0, 1), (8, 8, 8)])
def test_append_strides_and_positions(cuda, off, st_t, st_h):
    """Element loads where addresses or strides are not multiples of 16 bytes; given positions."""
    r = np.random.default_rng(off + 2 * st_t + 5 * st_h)
    D, heads, T = 128, 2, 5
    st = Setup(cuda, r, [T], [T], heads, D, 16)
    sh = D + st_h
    stt = 3 * heads * sh + st_t
    buf = torch.randn(off + T * stt + 16, device=cuda).to(torch.bfloat16)
    part = lambda i: buf[off + i * heads * sh:].as_strided((T, heads, D), (stt, sh, 1), off + i * heads * sh)  # noqa: E731
    q, k, v = part(0), part(1), part(2)
    pos = r.permutation(50)[:T].astype(np.int32)
    tab = r.standard_normal((50, D)).astype(np.float32)
    qo = kv4.append(q, k, v, st.cache, *st.args, rope=t(tab, cuda), positions=t(pos, cuda))
    kc, vc, kw, vw = ok.split_block(st.cache.cpu().numpy(), 16, D)
    for i in range(T):
        p = st.bt[0, 0]
        c, s, z = ok.quantize(ok.rotate(k[i].float().cpu().numpy(), tab[pos[i]], D, False, None))
        assert (kc[p, :, i] == c).all() and (kw[p, :, i] == ok.words(s, z)).all()
        c, s, z = ok.quantize(v[i].float().cpu().numpy())
        assert (vc[p, :, i] == c).all() and (vw[p, :, i] == ok.words(s, z)).all()
        want = torch.from_numpy(ok.rotate(q[i].float().cpu().numpy(), tab[pos[i]], D, False, None)).bfloat16()
        assert torch.equal(qo[i].cpu(), want)


def test_append_extremes(cuda):
    """Zeros, one-sided vectors, tiny, huge, NaN and infinite ones; and what is read back of them."""
    D, heads = 64, 1
    rows = [np.zeros(D), np.full(D, 3.0), np.full(D, -2.0), np.r_[1.0, np.zeros(D - 1)],
            np.linspace(-1, 1, D) * 1e-37, np.linspace(-1, 1, D) * 3e38, np.r_[np.nan, np.ones(D - 1)],
            np.r_[np.ones(D - 1), np.inf], np.linspace(0, 1, D) * 3e38, np.r_[-np.inf, np.ones(D - 1)]]
    x = torch.tensor(np.array(rows), dtype=torch.float32).bfloat16()[:, None]
    n = len(rows)
    st = Setup(cuda, np.random.default_rng(0), [n], [n], heads, D, 16)
    kv4.append(None, x.to(cuda), x.to(cuda).flip(-1), st.cache, *st.args)
    kc, vc, kw, vw = ok.split_block(st.cache.cpu().numpy(), 16, D)
    p = st.bt[0, 0]
    c, s, z = ok.quantize(x.float().numpy()[:, 0])
    w = ok.words(s, z)
    assert (kc[p, 0, :n] == c).all() and (kw[p, 0, :n] == w).all()
    assert (vc[p, 0, :n] == c[:, ::-1]).all() and (vw[p, 0, :n] == w).all()
    k, v = kv4.gather(st.cache, *st.args, tokens=n, head_dim=D, dtype=torch.float32)
    want = ok.values(c, w, np.float32)
    assert np.array_equal(k[:, 0].cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[[5, 6, 7, 9]]).all() and np.isfinite(want[[0, 1, 2, 3, 4, 8]]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 32)])
def test_gather_values(cuda, D, P, dtype):
    r = np.random.default_rng(D)
    st = Setup(cuda, r, [3, 0, 70], [3, 9, 70], 3, D, P)
    st.fill(r)
    k, v = kv4.gather(st.cache, *st.args, tokens=st.T, head_dim=D, dtype=dtype)
    for b in (0, 2):
        hk, hv, _, _ = st.host(b)
        s = slice(st.start[b], st.start[b + 1])
        # fp32 products of the scale and a whole number, then one rounding
        for got, w in ((k[s], hk), (v[s], hv)):
            w = torch.from_numpy(np.moveaxis(w, 1, 0).astype(np.float32)).to(dtype)
            assert torch.equal(got.cpu(), w)


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("D,P,heads,g,dtype,new,kv,causal,window,sinks", [
    (128, 16, 1, 1, "bf16", [1], [1], True, 0, 0),
    (128, 64, 2, 4, "bf16", [1, 1, 1], [17, 200, 64], True, 0, 0),
    (128, 32, 2, 8, "fp16", [1, 1], [129, 500], True, 0, 0),
    (64, 16, 3, 1, "fp16", [1, 1, 1], [5, 16, 333], True, 0, 0),
    (256, 64, 1, 6, "bf16", [1, 2], [70, 130], True, 0, 0),
    (128, 64, 1, 5, "fp16", [3, 7], [90, 260], True, 0, 0),
    (128, 128, 2, 3, "bf16", [5, 1, 0, 2], [5, 300, 40, 129], True, 0, 0),
    (64, 64, 1, 2, "bf16", [40], [100], True, 0, 0),
    (256, 16, 1, 2, "fp16", [9], [77], True, 0, 0),
    (128, 64, 1, 4, "bf16", [1, 1], [400, 65], True, 64, 4),
    (128, 16, 1, 4, "fp16", [6, 3], [300, 50], True, 20, 3),
    (64, 32, 1, 8, "fp16", [2], [500], True, 1, 0),
    (128, 64, 1, 2, "bf16", [4], [600], True, 100, 200),
    (128, 64, 1, 2, "bf16", [4], [600], True, 1000, 4),
    (256, 32, 1, 3, "bf16", [1, 30], [200, 31], True, 13, 1),
    (128, 64, 2, 2, "fp16", [3, 4], [100, 4], False, 0, 0),
    (128, 64, 1, 17, "bf16", [1, 2], [100, 40], True, 0, 0),
    (128, 64, 1, 40, "fp16", [1], [300], True, 0, 0),
    (128, 64, 2, 1, "fp16", [9, 1, 1, 1], [200, 70, 1, 400], True, 0, 0),
    (256, 32, 2, 2, "fp16", [1, 1], [300, 70], True, 0, 0),
    (256, 64, 1, 2, "fp16", [3, 1], [900, 70], True, 60, 4),
])
def test_attention(cuda, D, P, heads, g, dtype, new, kv, causal, window, sinks):
    r = np.random.default_rng(D + P + sum(kv) + window)
    st = Setup(cuda, r, new, kv, heads, D, P, extra=2)
    st.fill(r)
    T = st.T + 3
    wide = torch.from_numpy(r.standard_normal((T, 2 * heads * g, D)) * 2).to(cuda, DT[dtype])
    q = wide[:, heads * g:]                                  # strided
    out = torch.full((T, heads * g, D), 5.0, dtype=DT[dtype], device=cuda)
    lse = torch.full((T, heads * g), 5.0, device=cuda)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    scale = 0.7 * D ** -0.5
    kv4.attend(q, st.cache, *st.args, scale=scale, causal=causal, window=window, sinks=sinks, out=out, lse=lse,
               info=info)
    assert info.item() == 0
    check_attention(st, q, out, scale, causal, window, sinks, lse)
    assert (out[st.T:] == 5).all() and (lse[st.T:] == 5).all()


def test_attention_empty_rows(cuda):
    """Queries in front of a sequence's first token, and sequences without tokens, give 0 and -inf."""
    r = np.random.default_rng(3)
    st = Setup(cuda, r, [4, 2, 3], [2, 0, 3], 2, 128, 16)
    st.fill(r)
    q = torch.randn(st.T, 4, 128, device=cuda).bfloat16()
    lse = torch.empty(st.T, 4, device=cuda)
    out = kv4.attend(q, st.cache, *st.args, lse=lse)
    check_attention(st, q, out, 128 ** -0.5, lse=lse)
    assert (lse[:2] == -np.inf).all() and (out[4:6] == 0).all()


@pytest.mark.parametrize("D,P,heads,g,dtype,B,n,L,window,sinks", [
    (128, 64, 2, 4, "bf16", 1, 1, 20011, 0, 0),
    (128, 128, 1, 8, "fp16", 2, 1, 33000, 0, 0),
    (64, 16, 1, 1, "bf16", 3, 1, 9000, 0, 0),
    (256, 32, 1, 4, "bf16", 1, 2, 7001, 0, 0),
    (128, 64, 2, 4, "bf16", 2, 1, 30000, 9000, 100),
    (128, 64, 1, 4, "fp16", 300, 1, 150, 0, 0),
    (64, 64, 1, 2, "fp16", 3000, 1, 7, 0, 0),
    (128, 64, 1, 4, "bf16", 2, 5, 12345, 0, 0),
    (128, 64, 2, 4, "fp16", 40, 1, 9000, 0, 0),
    (64, 32, 2, 2, "bf16", 33, 2, 6000, 1500, 4),
    (256, 64, 2, 2, "fp16", 50, 1, 3000, 0, 0),
])
def test_attention_long_and_many(cuda, D, P, heads, g, dtype, B, n, L, window, sinks):
    """Split sequences, and more sequences than a block has threads."""
    r = np.random.default_rng(L)
    kv = [max(n, L - 97 * (b % 5) if L > 1000 else L - b % 7) for b in range(B)]
    st = Setup(cuda, r, [n] * B, kv, heads, D, P)
    st.fill_fast(torch.Generator(cuda).manual_seed(L))
    q = torch.from_numpy(r.standard_normal((st.T, heads * g, D))).to(cuda, DT[dtype])
    lse = torch.empty(st.T, heads * g, device=cuda)
    out = kv4.attend(q, st.cache, *st.args, window=window, sinks=sinks, lse=lse)
    seqs = sorted({0, 1 % B, B // 2, B - 1})
    check_attention(st, q, out, D ** -0.5, True, window, sinks, lse, seqs=seqs)


@pytest.mark.parametrize("D,P,heads,g,dtype,new,kv,causal,window,sinks", [
    (128, 64, 2, 4, "bf16", [700, 130], [1500, 130], True, 0, 0),
    (128, 16, 1, 8, "fp16", [257], [1000], True, 0, 0),
    (64, 32, 1, 3, "bf16", [511, 1, 90], [511, 700, 1201], True, 0, 0),
    (256, 64, 1, 2, "fp16", [300], [900], True, 0, 0),
    (128, 64, 1, 4, "bf16", [600], [2000], True, 100, 7),
    (256, 128, 1, 4, "bf16", [200, 65], [1111, 300], True, 300, 130),
    (64, 64, 2, 1, "fp16", [400], [1300], True, 64, 0),
    (128, 64, 1, 2, "fp16", [200, 33], [500, 40], False, 0, 0),
    (128, 256, 1, 1, "bf16", [300, 0, 200], [300, 50, 100], True, 0, 0),
    # wide heads, a few steps and many; one row behind a tile
    (256, 64, 2, 4, "bf16", [33, 64, 65], [33, 64, 129], True, 0, 0),
    (256, 16, 1, 4, "fp16", [300, 200], [2000, 2100], True, 64, 0),
    (256, 64, 1, 8, "bf16", [129], [3000], True, 1024, 16),
    (64, 128, 1, 16, "bf16", [17, 33], [64, 2049], True, 0, 0),
    # new tokens of decoding sequences beside a prompt's, some without any key
    (128, 64, 2, 4, "bf16", [1, 300, 1, 2, 4], [700, 900, 33, 2000, 2], True, 0, 0),
    (128, 32, 2, 4, "fp16", [1, 300, 1, 2, 4], [700, 900, 33, 2000, 0], True, 50, 3),
])
def test_attention_prompts(cuda, D, P, heads, g, dtype, new, kv, causal, window, sinks):
    """Many query rows per key."""
    r = np.random.default_rng(sum(kv))
    st = Setup(cuda, r, new, kv, heads, D, P)
    st.fill_fast(torch.Generator(cuda).manual_seed(sum(kv)))
    T = st.T + 5
    q = torch.from_numpy(r.standard_normal((T, heads * g, D))).to(cuda, DT[dtype])
    out = torch.full((T, heads * g, D), 5.0, dtype=DT[dtype], device=cuda)
    lse = torch.full((T, heads * g), 5.0, device=cuda)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    kv4.attend(q, st.cache, *st.args, causal=causal, window=window, sinks=sinks, out=out, lse=lse, info=info)
    assert info.item() == 0
    rows = [0, 1, 2, 29, 31, 32, 33, 63, 64, 65, 127, 128, 200, 255, 256, 399, 510, 599, 699]
    check_attention(st, q, out, D ** -0.5, causal, window, sinks, lse, rows=rows)
    assert (out[st.T:] == 5).all() and (lse[st.T:] == 5).all()


@pytest.mark.parametrize("new,g", [(1, 4), (96, 4)])
def test_attention_ranges(cuda, new, g):
    """Very large and very small queries, keys and values, and values whose scales differ by 10^8."""
    r = np.random.default_rng(5)
    D, L = 128, 256
    st = Setup(cuda, r, [new], [L], 1, D, 64)
    raw = st.cache.cpu().numpy()
    for j in range(L):
        x = r.standard_normal((2, D))
        x[0] *= 1e-6
        x[1] *= 10.0 ** (-4 + 8 * (j % 9) / 8)
        c, s, z = ok.quantize(x)
        w = ok.words(s, z)
        for i in (0, 1):
            ok.put(raw[st.bt[0, j // 64], 0], 64, D, j % 64, c[i], w[i], i)
    st.cache.copy_(torch.from_numpy(raw))
    q = torch.from_numpy(r.standard_normal((new, g, D)) * 1e6 * np.array([1, 0.1, 1e-9, 3])[None, :, None]).to(
        cuda, torch.bfloat16)
    out = kv4.attend(q, st.cache, *st.args, scale=0.1)
    check_attention(st, q, out, 0.1, rows=[0, 40, 95])


@pytest.mark.parametrize("new", [1, 80])
def test_attention_nan_stays_in_its_rows(cuda, new):
    """A NaN token is seen by the rows that see it and by no other; a NaN query spoils its own row."""
    r = np.random.default_rng(6)
    st = Setup(cuda, r, [new, new], [200, 200], 1, 128, 64)
    st.fill(r)
    x = torch.randn(400, 1, 128, device=cuda).bfloat16()
    bad = x[:1].clone()
    bad[0, 0, 5] = float("nan")
    # sequence 0: token 150 is NaN; windows of 40 (and sinks 2) leave rows that do not see it
    one = (st.args[0][:1], i32([0, 1], cuda), i32([151], cuda))
    kv4.append(None, bad, bad, st.cache, *one)
    q = torch.randn(2 * new, 2, 128, device=cuda).bfloat16()
    q[new, 1] = float("nan")
    out = f64(kv4.attend(q, st.cache, *st.args, window=40, sinks=2))
    for i in range(new):
        p = 200 - new + i
        sees = p >= 150 and 150 > p - 40
        assert np.isnan(out[i]).all() == sees and np.isnan(out[i]).any() == sees, i
    assert np.isnan(out[new, 1]).all() and np.isfinite(out[new, 0]).all() and np.isfinite(out[new + 1:]).all()


@pytest.mark.parametrize("new", [1, 70])
def test_bad_pages_and_lengths(cuda, new):
    """Pages outside the cache, lengths beyond the table, rows beyond the tensor: noticed, nothing else harmed."""
    r = np.random.default_rng(7)
    st = Setup(cuda, r, [new, new], [200, 300], 2, 128, 64)
    st.fill(r)
    q = torch.randn(st.T, 4, 128, device=cuda).bfloat16()
    good = kv4.attend(q, st.cache, *st.args)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    bt = st.bt.copy()
    bt[0, 1] = st.pages
    bad = (t(bt, cuda),) + st.args[1:]
    out = kv4.attend(q, st.cache, *bad, info=info)
    assert info.item() == -1 and torch.equal(out[new:], good[new:])
    # keys of the bad page are keys nobody sees
    hk, hv, _, _ = st.host(0)
    keep = np.r_[0:64, 128:200]
    o, _, _ = ok.attend(f64(q)[0, 0], hk[0][keep], hv[0][keep], 128 ** -0.5,
                        ok.visible(200 - new, 200, True, 0, 0)[keep])
    assert np.abs(f64(out)[0, 0] - o).max() <= 0.01
    for change in ((st.args[0], st.args[1], i32([200, 10 ** 6], cuda)), (st.args[0], st.args[1], i32([200, -5], cuda)),
                   (st.args[0], i32([0, new, 10 * new], cuda), st.args[2]),
                   (st.args[0], i32([0, new, -3], cuda), st.args[2])):
        info.zero_()
        out = kv4.attend(q, st.cache, *change, info=info)
        torch.cuda.synchronize()
        assert info.item() == -1 and torch.equal(out[:new], good[:new])
    # append: a page outside the cache, a position outside the table
    before = st.cache.clone()
    x = torch.randn(st.T, 2, 128, device=cuda).bfloat16()
    nowhere = torch.full_like(st.args[0], -1)
    info.zero_()
    kv4.append(None, x, x, st.cache, nowhere, *st.args[1:], info=info)
    assert info.item() == -1 and torch.equal(st.cache, before)
    info.zero_()
    kv4.append(None, x, x, st.cache, *st.args, rope=torch.zeros(10, 128, device=cuda), info=info)
    assert info.item() == -1 and torch.equal(st.cache, before)
    info.zero_()
    kv4.append(None, x, x, st.cache, *st.args, positions=torch.full((st.T,), -1, dtype=torch.int32, device=cuda),
               rope=torch.zeros(1000, 128, device=cuda), info=info)
    assert info.item() == -1 and torch.equal(st.cache, before)
    info.zero_()
    k = torch.full((st.T, 2, 128), 5.0, device=cuda)
    abi.kronq_kv4_gather(st.cache, nowhere, *st.args[1:], k, k.clone(), info)
    assert info.item() == -1 and (k == 5).all()


def test_window_pages_may_be_gone(cuda):
    """Table entries of pages that no query sees are not looked at."""
    r = np.random.default_rng(8)
    st = Setup(cuda, r, [2], [1000], 1, 128, 16)
    st.fill(r)
    q = torch.randn(2, 4, 128, device=cuda).half()
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    bt = st.bt.copy()
    bt[0, 1:54] = 10 ** 6                 # sinks: page 0; the window begins with token 899 (page 56)
    out = kv4.attend(q, st.cache, t(bt, cuda), *st.args[1:], window=100, sinks=5, info=info)
    assert info.item() == 0
    check_attention(st, q, out, 128 ** -0.5, True, 100, 5)


@pytest.mark.parametrize("new", [1, 90])
def test_same_bits_again(cuda, new):
    r = np.random.default_rng(9)
    st = Setup(cuda, r, [new] * 3, [5000, 100, 3000], 2, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(1))
    q = torch.randn(st.T, 8, 128, device=cuda).bfloat16()
    a = kv4.attend(q, st.cache, *st.args)
    for _ in range(3):
        assert torch.equal(a, kv4.attend(q, st.cache, *st.args))


def test_two_streams(cuda):
    """Two calls at once, each with the workspace the call allocates."""
    r = np.random.default_rng(10)
    st = [Setup(cuda, r, [1, 60][i:i + 1], [9000], 2, 128, 64) for i in (0, 1)]
    qs, want = [], []
    for i, s in enumerate(st):
        s.fill_fast(torch.Generator(cuda).manual_seed(i))
        qs.append(torch.randn(s.T, 8, 128, device=cuda).bfloat16())
        want.append(kv4.attend(qs[i], s.cache, *s.args))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(kv4.attend(qs[i], st[i].cache, *st[i].args, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_decode_loop_in_a_graph(cuda):
    """A prompt, then tokens one by one: append and attend captured once and replayed with the
    lengths moving on; a second graph of a window layer is replayed in between.  Against fp64
    attention over the values read back."""
    r = np.random.default_rng(11)
    D, P, heads, g, n0, steps = 128, 16, 2, 4, [37, 20], 30
    kvmax = [x + steps for x in n0]
    st = Setup(cuda, r, [1, 1], kvmax, heads, D, P)
    tab = kv4.rope_table(128, D, device=cuda)
    sg = t((1 - 2 * r.integers(0, 2, D)).astype(np.int8), cuda)
    new = lambda T: torch.randn(T, (g + 2) * heads, D, device=cuda).bfloat16()  # noqa: E731
    parts = lambda x: (x[:, :g * heads], x[:, g * heads:(g + 1) * heads], x[:, (g + 1) * heads:])  # noqa: E731
    x = new(sum(n0))
    start = i32([0, n0[0], sum(n0)], cuda)
    lens = i32(n0, cuda)
    q = kv4.append(*parts(x), st.cache, st.args[0], start, lens, rope=tab, signs=sg)
    o = kv4.attend(q, st.cache, st.args[0], start, lens)
    st.kv, st.new, st.start = n0, n0, [0, n0[0]]
    check_attention(st, q, o, D ** -0.5)
    # one token per step
    x1, start1 = new(2), i32([0, 1, 2], cuda)

    def step(window):
        q = kv4.append(*parts(x1), st.cache, st.args[0], start1, lens, rope=tab, signs=sg)
        return q, kv4.attend(q, st.cache, st.args[0], start1, lens, window=window, sinks=2 if window else 0)

    lens += 1
    step(0), step(9)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (0, 9):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(window))
        graphs.append(gr)
    st.new, st.start = [1, 1], [0, 1]
    for i in range(1, steps):
        x1.copy_(new(2))
        if i > 1:
            lens += 1
        for gr in graphs:
            gr.replay()
        st.kv = [x + i for x in n0]
        if i in (1, 2, 11, 12, steps - 1):
            for (q, o), window in zip(outs, (0, 9)):
                check_attention(st, q, o, D ** -0.5, True, window, 2 if window else 0)


@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_unaligned(cuda, new, dtype):
    """Queries that no 16-byte load fits, outputs on 8-byte boundaries, rows apart."""
    r = np.random.default_rng(20 + new)
    st = Setup(cuda, r, [new, 2], [400, 130], 2, 128, 64)
    st.fill(r)
    T, H, D = st.T, 6, 128
    q = torch.randn(1 + T * H * (D + 1), device=cuda).to(dtype)[1:].view(T, H, D + 1)[..., :D]
    buf = torch.full((4 + T * (H * (D + 4) + 8),), 3.0, dtype=dtype, device=cuda)
    out = buf.as_strided((T, H, D), (H * (D + 4) + 8, D + 4, 1), 4)
    kv4.attend(q, st.cache, *st.args, out=out)
    check_attention(st, q, out, D ** -0.5)
    out.fill_(3.0)
    assert (buf == 3).all()                        # nothing between the rows was written


@pytest.mark.parametrize("new", [1, 100])
def test_shared_pages(cuda, new):
    """Two sequences over the same pages (a shared prompt), each with its own length."""
    r = np.random.default_rng(21)
    st = Setup(cuda, r, [new, new], [3000, 2500], 2, 128, 64)
    st.bt[1, :40] = st.bt[0, :40]
    st.args = (t(st.bt, cuda),) + st.args[1:]
    st.fill_fast(torch.Generator(cuda).manual_seed(2))
    q = torch.randn(st.T, 8, 128, device=cuda).half()
    check_attention(st, q, kv4.attend(q, st.cache, *st.args), 128 ** -0.5, rows=[0, 50, 99])


@pytest.mark.parametrize("new,n", [(2, 150), (64, 150), (200, 10)])
def test_overlapping_rows(cuda, new, n):
    """Many sequences that claim the same rows ask for more blocks than the grid has: noticed, and
    nothing outside the output is touched (a workspace full of large numbers leads nowhere)."""
    r = np.random.default_rng(22)
    L = 4000
    st = Setup(cuda, r, [new], [L], 1, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(3))
    q = torch.randn(new, 4, 128, device=cuda).bfloat16()
    start = np.zeros(2 * n, dtype=np.int32)
    start[1::2] = new                              # every second sequence has the rows, the others fewer than none
    bt = np.repeat(st.bt, 2 * n - 1, 0)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    need = abi.kronq_kv4_attention_workspace_size(new, 4, 1, 128, 2 * n - 1)
    ws = torch.full((need + 4096,), 127, dtype=torch.uint8, device=cuda)
    out = torch.full((new + 2, 4, 128), 5.0, dtype=torch.bfloat16, device=cuda)
    kv4.attend(q, st.cache, t(bt, cuda), t(start, cuda), i32([L] * (2 * n - 1), cuda), out=out[:new],
               ws=ws[:-4096], info=info)
    torch.cuda.synchronize()
    assert info.item() == -1 and (ws[-4096:] == 127).all() and (out[new:] == 5).all()


def test_merging_by_log_sum_exp(cuda):
    """A shared prefix seen in full and the rest seen causally join to one causal attention."""
    r = np.random.default_rng(12)
    st = Setup(cuda, r, [3], [300], 1, 128, 64)
    st.fill(r)
    q = torch.randn(3, 4, 128, device=cuda).half()
    lse = [torch.empty(3, 4, device=cuda) for _ in range(3)]
    whole = kv4.attend(q, st.cache, *st.args, lse=lse[0])
    a = kv4.attend(q, st.cache, st.args[0], st.args[1], i32([128], cuda), causal=False, lse=lse[1])
    b = kv4.attend(q, st.cache, st.args[0][:, 2:], st.args[1], i32([172], cuda), lse=lse[2])
    w = torch.softmax(torch.stack(lse[1:]).double(), 0)[..., None]
    got = w[0] * a.double() + w[1] * b.double()
    # three results, each off by a rounding of its fp16 output and of its probabilities
    assert (got - whole.double()).abs().max().item() <= 4 * 2.0 ** -11 * 12
    assert (torch.logsumexp(torch.stack(lse[1:]), 0) - lse[0]).abs().max().item() <= 1e-4


def test_refuses_another_device_and_small_workspaces(cuda):
    r = np.random.default_rng(13)
    st = Setup(cuda, r, [1], [20], 1, 128, 16)
    q = torch.randn(1, 4, 128, device=cuda).bfloat16()
    with pytest.raises(ValueError):
        kv4.attend(q.cpu(), st.cache, *st.args)
    with pytest.raises(ValueError):
        kv4.attend(q, st.cache, st.args[0].cpu(), *st.args[1:])
    with pytest.raises(abi.KronqError):
        kv4.attend(q, st.cache, *st.args, ws=torch.empty(256, dtype=torch.uint8, device=cuda))
    with pytest.raises(abi.KronqError):
        kv4.attend(q[:, :3].contiguous().repeat(1, 1, 1), kv4.make_cache(2, 16, 2, 128, cuda), *st.args)
