"""Attention over the 4-bit cache where numbers are far apart: value and key scales, one key
that holds nearly all of the probability, fp16 outputs whose parts cancel.

Every output element is compared with fp64 attention of the cached values.  With p the exact
probabilities, s the value scales, V = s (c - z) the cached values (|c - z| <= 15) and o the
exact output, of the keys j that the row sees:

  |err| <= eps/2 |o|                                the output's rounding
         + sum_j p_j |V_j| (t + u_j) + |o| sum_j p_j u_j
         + 15 n 2^-floor max_j p_j s_j              weights that fp16 holds as subnormals
         + Ea 30 sum_j p_j s_j                      sums of codes and of zero points

t: roundings of a weight p s to fp16 (2^-11 for one term, 2^-21 for two), with bf16 queries of
the many-rows kernel also of the value: 3 times 2^-11.
u_j: what a probability is off by: its score by 2 D 2^-23 scale sum|q| 15 k_j (sums of codes and of
zero points; keys in fp16: and 2^-11 scale sum |q_d k_jd|), 2^-22 for the exponential, and 2^-23
of every number of binary digits that a score, or its distance from the maximum and the value
scale's exponent, is away from 0.
floor: an fp16 subnormal is off by 2^-25 where the row's largest weight is at least 2^(floor - 25).
Ea: 2^-23 for each 16 keys with a weight that is not 0 and 64 for joins.
"""

import numpy as np
import pytest
import torch

import kv4_cases
from gpu_helpers import t
from oracle import kv4 as ok
from post_quantization_02_b200 import kv4
from test_gpu_kv4 import DT, Setup, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def own_random_numbers(cuda):
    """The same inputs whatever ran before, and none taken from what runs behind."""
    with torch.random.fork_rng(devices=[cuda]):
        torch.manual_seed(2024)
        yield


def words_of(scale, zero=0):
    return ok.words(np.asarray([scale], dtype=np.float32).view(np.uint32).__and__(np.uint32(0xFFFFFFF0)).view(
        np.float32), np.asarray([zero], dtype=np.uint8))[0]


class Bytes:
    """A setup's cache on the host, written token by token."""

    def __init__(self, st):
        self.st, self.raw = st, st.cache.cpu().numpy()

    def put(self, b, j, h, vec, isv):
        st = self.st
        c, s, z = ok.quantize(np.asarray(vec)[None])
        ok.put(self.raw[st.bt[b, j // st.P], h], st.P, st.D, j % st.P, c[0], ok.words(s, z)[0], isv)

    def done(self):
        self.st.cache.copy_(torch.from_numpy(self.raw))


def check(st, q, out, scale, terms, floor, causal=True, window=0, sinks=0, lse=None, rows=None, keys_rounded=False,
          seqs=None):
    eps = torch.finfo(q.dtype).eps
    qh, oh = f64(q), f64(out)
    g = q.shape[1] // st.heads
    tt = {1: 2.0 ** -11, 2: 2.0 ** -21, 3: 3 * 2.0 ** -11}[terms]
    for b in range(len(st.kv)) if seqs is None else seqs:
        k, v, ks, vs = st.host(b)
        L = st.kv[b]
        for i in range(st.new[b]) if rows is None else rows:
            mask = ok.visible(L - st.new[b] + i, L, causal, window, sinks)
            row = st.start[b] + i
            for h in range(q.shape[1]):
                kh = h // g
                kk, vv, sk, sv = k[kh][mask], v[kh][mask], ks[kh][mask], vs[kh][mask]
                a = scale * (kk @ qh[row, h])
                e = np.exp(a - a.max())
                p = e / e.sum()
                o = p @ vv
                qa = np.abs(qh[row, h])
                ex = 2 * st.D * 2.0 ** -23 * scale * qa.sum() * 15 * sk
                if keys_rounded:
                    ex = ex + scale * 2.0 ** -11 * (np.abs(kk) @ qa)
                digits = 1.45 * (2 * np.abs(a) + 2 * np.abs(a - a.max())) + 40 + np.abs(np.log2(sv)).max()
                u = ex + 2.0 ** -22 + 2.0 ** -23 * digits
                w = p * sv
                used = np.add.reduceat(w > w.max() * 2.0 ** -40, np.arange(0, len(w), 16)) > 0
                ea = 2.0 ** -23 * (64 + used.sum())
                tol = (eps / 2 * np.abs(o) + (p * (tt + u)) @ np.abs(vv) + np.abs(o) * (p @ u)
                       + 15 * len(w) * 2.0 ** -floor * w.max() + ea * 30 * w.sum() + torch.finfo(q.dtype).tiny)
                bad = ~(np.abs(oh[row, h] - o) <= tol)
                assert not bad.any(), (b, i, h, oh[row, h][bad][:4], o[bad][:4], tol[bad][:4])
                if lse is not None:
                    want = a.max() + np.log(e.sum())
                    assert abs(lse[row, h].item() - want) <= (p @ u) + 2.0 ** -20 * (1 + abs(want)), (b, i, h)


def few(T, g, B, D, dtype="bf16"):
    return T * g <= (40 if D == 256 and dtype == "fp16" else 64) * B


@pytest.mark.parametrize("dtype,big", [("fp16", 6e4), ("bf16", 1e5), ("bf16", 1e12), ("bf16", 3e38)])
@pytest.mark.parametrize("D,new,g", [(128, 3, 4), (64, 3, 1), (256, 2, 4), (128, 5, 8), (128, 130, 4), (64, 300, 1),
                                     (256, 70, 2)])
def test_values_far_apart(cuda, D, new, g, dtype, big):
    """Value vectors that are very large, seen by some rows and masked for others: exact enough for
    both, and finite."""
    r = np.random.default_rng(D + new)
    L, window, sinks = new + 200, 90, 3
    st = Setup(cuda, r, [new], [L], 1, D, 64)
    st.fill(r)
    w = Bytes(st)
    where = (1, L - 1, L - new - 60, L - new // 2 - 1, L - new - 95)
    for j in where:
        x = np.linspace(0, 1, D) * big
        w.put(0, j, 0, x[::-1] if j & 1 else x, 1)
    w.done()
    q = torch.from_numpy(r.standard_normal((st.T, g, D))).to(cuda, DT[dtype])
    is_few = few(new, g, 1, D, dtype)
    rows = range(new) if new < 20 else [0, 1, 4, 5, 31, 33, 59, 60, 61, new // 2 - 1, new // 2, new - 2, new - 1]
    for win, snk in ((0, 0), (window, sinks), (window, 0), (1, 0)):
        lse = torch.empty(st.T, g, device=cuda)
        out = kv4.attend(q, st.cache, *st.args, window=win, sinks=snk, lse=lse)
        terms = (2 if dtype == "fp16" else 1) if is_few else (1 if dtype == "fp16" else 3)
        # (many rows: scales of the same 64 keys up to 2^8 apart share a factor)
        check(st, q, out, D ** -0.5, terms, 33 if is_few else 25, window=win, sinks=snk, lse=lse, rows=rows,
              keys_rounded=not is_few and dtype == "bf16")


@pytest.mark.parametrize("D,new,g", [(128, 2, 4), (128, 130, 4), (64, 300, 1), (256, 70, 2)])
def test_keys_far_apart(cuda, D, new, g):
    """A key far larger than its neighbours, seen by some rows only, leaves the others' scores alone."""
    r = np.random.default_rng(D)
    L = new + 100
    for big in (1e6, 1e15):
        st = Setup(cuda, r, [new], [L], 1, D, 64)
        st.fill(r)
        w = Bytes(st)
        q = r.standard_normal((st.T, g, D))
        for j in (L - 1, L - new // 2 - 1):
            x = r.standard_normal(D)
            x -= q[-1, 0] * (x @ q[-1, 0]) / (q[-1, 0] @ q[-1, 0])
            w.put(0, j, 0, x * big, 0)
        w.done()
        qt = torch.from_numpy(q).to(cuda, torch.bfloat16)
        out = kv4.attend(qt, st.cache, *st.args)
        is_few = few(new, g, 1, D)
        check(st, qt, out, D ** -0.5, 1 if is_few else 3, 33 if is_few else 25, keys_rounded=not is_few,
              rows=range(new // 2) if new < 20 else [0, 1, 31, new // 2 - 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,g", [(1, 4), (1, 1), (2, 8), (20, 4)])
@pytest.mark.parametrize("first", [1e-6, 1.0, 0.0])
def test_one_key_holds_the_probability(cuda, dtype, new, g, first):
    """The first key is 17 nats above all others (a sink), its value near zero or like theirs: what the
    tens of thousands of others add is not lost.  (Many sequences over the same pages: a block then
    takes all of a sequence's keys.)"""
    L, D, P, B, heads = 30000, 128, 64, 160, 4
    r = np.random.default_rng(40)
    st = Setup(cuda, r, [new], [L], heads, D, P)
    n = st.pages * heads
    c = torch.randint(0, 256, (n, P * D // 2), generator=torch.Generator(cuda).manual_seed(3), device=cuda,
                      dtype=torch.int32).to(torch.uint8)
    word = lambda s: int(words_of(s))  # noqa: E731
    st.cache.zero_()
    blk = st.cache.view(n, P * (D + 8))
    blk[:, P * D // 2:P * D] = c
    blk[:, P * D:].view(torch.int32).view(n, 2, P).copy_(
        torch.tensor([word(1.0), word(0.13)], dtype=torch.int32, device=cuda)[:, None].expand(n, 2, P))
    w = Bytes(st)
    for h in range(heads):
        w.put(0, 0, h, np.full(D, 17.0), 0)
        w.put(0, 0, h, r.random(D) * first, 1)
    w.done()
    st.new, st.kv, st.T = [new] * B, [L] * B, new * B
    st.bt, st.start = np.repeat(st.bt, B, 0), new * np.arange(B + 1, dtype=np.int32)
    batch = (t(st.bt, cuda), t(st.start, cuda), torch.full((B,), L, dtype=torch.int32, device=cuda))
    q = torch.ones(st.T, heads * g, D, device=cuda).to(DT[dtype])
    lse = torch.empty(st.T, heads * g, device=cuda)
    out = kv4.attend(q, st.cache, *batch, scale=1 / D, lse=lse)
    is_few = few(new, g, 1, D, dtype)
    terms = (2 if dtype == "fp16" else 1) if is_few else (1 if dtype == "fp16" else 3)
    check(st, q, out, 1 / D, terms, 33, lse=lse, rows=[new - 1], seqs=[0, B - 1],
          keys_rounded=not is_few and dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,g", [(1, 4), (3, 8), (100, 4)])
def test_zero_and_tiny_values(cuda, dtype, new, g):
    """Zero vectors count in the sum of probabilities; a whole sequence of zero or of tiny values."""
    r = np.random.default_rng(41)
    D = 128
    st = Setup(cuda, r, [new] * 3, [300, 280, 290], 1, D, 64)
    st.fill(r)
    w = Bytes(st)
    for j in range(300):
        if j % 3 or 64 <= j < 128:
            w.put(0, j, 0, np.zeros(D), 1)
        if j < 280:
            w.put(1, j, 0, np.zeros(D), 1)
        if j < 290:
            w.put(2, j, 0, r.standard_normal(D) * 1e-25, 1)
    w.done()
    q = torch.from_numpy(r.standard_normal((st.T, g, D)) * 3).to(cuda, DT[dtype])
    lse = torch.empty(st.T, g, device=cuda)
    out = kv4.attend(q, st.cache, *st.args, lse=lse)
    is_few = few(st.T, g, 3, D, dtype)
    terms = (2 if dtype == "fp16" else 1) if is_few else (1 if dtype == "fp16" else 3)
    # (scales below 2^-80 lie lower in fp16's range: these are at 2^-86)
    check(st, q, out, D ** -0.5, terms, 28, lse=lse, rows=[0, 1 % new, new - 1],
          keys_rounded=not is_few and dtype == "bf16")
    st.new, st.kv, st.start = st.new[:2], st.kv[:2], st.start[:3]
    check(st, q, out, D ** -0.5, terms, 33, lse=lse, rows=[0, 1 % new, new - 1],
          keys_rounded=not is_few and dtype == "bf16")
    assert not out[new:2 * new].any()


@pytest.mark.parametrize("D,new,g,L", [(128, 1, 4, 2), (128, 1, 1, 3), (64, 1, 3, 2), (256, 1, 4, 2),   # 4 rows at most
                                       (128, 1, 8, 2), (128, 1, 7, 40), (256, 3, 6, 4), (64, 2, 3, 3),
                                       (128, 2, 8, 3), (64, 3, 5, 4), (128, 4, 16, 5),
                                       (128, 1, 4, 9000), (128, 1, 8, 9000), (128, 2, 8, 9000)])
def test_fp16_outputs_that_cancel(cuda, D, new, g, L):
    """fp16 outputs are as exact as their own rounding also where values cancel: two fp16 terms of each
    weight.  (One term alone is off by up to 2^-12 of each value, where the two largest differ in sign.)"""
    r = np.random.default_rng(D + L)
    st = Setup(cuda, r, [new] * 2, [max(L, new), max(L, new) + 1], 2, D, 64)
    st.fill(r) if L < 100 else st.fill_fast(torch.Generator(cuda).manual_seed(3))
    w = Bytes(st)
    for b in (0, 1):
        n = st.kv[b]
        x = r.standard_normal((2, D)) + 3
        for h in (0, 1):
            for j in range(n):
                # all but the last few keys are far below: they add nothing
                k = r.standard_normal(D) * 0.1 if j >= n - 4 else np.full(D, -90.0)
                if L < 100 or j >= n - 4:
                    w.put(b, j, h, k, 0)
                    w.put(b, j, h, x[h] if j % 2 else -x[h], 1)
            if L >= 100:
                # (keys far below, by their words alone: codes 0, zero point 15, scale 6)
                for m in range(-(-n // 64)):
                    blk = w.raw[st.bt[b, m], h]
                    keep = [j for j in range(n - 4, n) if j // 64 == m]
                    old = {j: (blk[(j % 64) * D // 2:(j % 64 + 1) * D // 2].copy(),
                               blk[64 * D + 4 * (j % 64):64 * D + 4 * (j % 64) + 4].copy()) for j in keep}
                    blk[:64 * D // 2] = 0
                    blk[64 * D:64 * D + 256] = np.full(64, words_of(6.0, 15), dtype=np.uint32).view(np.uint8)
                    for j, (c, wd) in old.items():
                        blk[(j % 64) * D // 2:(j % 64 + 1) * D // 2] = c
                        blk[64 * D + 4 * (j % 64):64 * D + 4 * (j % 64) + 4] = wd
    w.done()
    q = torch.from_numpy(np.abs(r.standard_normal((st.T, 2 * g, D))) + 0.5).to(cuda, torch.float16)
    out = kv4.attend(q, st.cache, *st.args)
    assert few(st.T, g, 2, D, "fp16")
    check(st, q, out, D ** -0.5, 2, 33)


@pytest.mark.parametrize("D,g,L,n", [(128, 4, 8, 8), (128, 1, 4, 4), (64, 3, 2, 2), (256, 4, 16, 16),     # 4 rows at most
                                     (128, 8, 8, 8), (256, 6, 4, 4), (64, 5, 16, 16),                    # 8
                                     (128, 16, 8, 8), (64, 12, 4, 4),                                    # 16
                                     (128, 4, 9000, 8), (128, 8, 9000, 16), (64, 16, 20000, 8), (256, 2, 9000, 8)])
def test_two_terms_of_a_weight(cuda, D, g, L, n):
    """fp16 outputs of pairs that cancel (kv4_cases.py: one fp16 term of each weight is beyond the
    bound), in a short sequence and spread over a long one whose other keys are far below."""
    r = np.random.default_rng(60 + D + g)
    heads, B, P = 4, 2, 64
    st = Setup(cuda, r, [1] * B, [L] * B, heads, D, P)
    raw = st.cache.cpu().numpy()
    far_code, far_scale, far_zero = kv4_cases.key_far_below()
    one = words_of(1.0)
    raw[:, :, :P * D // 2] = far_code
    raw[:, :, P * D:P * D + 4 * P] = np.full(P, words_of(far_scale, far_zero), np.uint32).view(np.uint8)
    raw[:, :, P * D + 4 * P:] = np.full(P, one, np.uint32).view(np.uint8)
    want = {}
    for b in range(B):
        for h in range(heads):
            s, z, c = kv4_cases.pairs(r, n, D)
            want[b, h] = (*kv4_cases.exact(s, z, c), s)
            at = np.sort(r.permutation(L)[:n])
            for j, i in zip(at, r.permutation(n)):
                blk = raw[st.bt[b, j // P], h]
                ok.put(blk, P, D, j % P, np.zeros(D, np.uint8), one, 0)
                ok.put(blk, P, D, j % P, c[i], ok.words(s[i:i + 1], z[i:i + 1])[0], 1)
    st.cache.copy_(torch.from_numpy(raw))
    q = torch.from_numpy(np.abs(r.standard_normal((B, heads * g, D))) + 0.5).to(cuda, torch.float16)
    out = f64(kv4.attend(q, st.cache, *st.args))
    for (b, h), (o, v, s) in want.items():
        tol = kv4_cases.bound(o, v, s, 2.0 ** -10) + 2.0 ** -25       # (outputs that fp16 holds as subnormals)
        for row in range(h * g, (h + 1) * g):
            bad = ~(np.abs(out[b, row] - o) <= tol)
            assert not bad.any(), (b, row, out[b, row][bad][:4], o[bad][:4], tol[bad][:4])
