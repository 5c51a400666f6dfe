"""The 4-bit key/value cache's calls on the GPU: streams, refusals, batches that contradict
themselves.  (What they compute: test_gpu_kv4.py.)"""

import numpy as np
import pytest
import torch

from gpu_helpers import t
from oracle import kv4 as ok
from post_quantization_02_b200 import abi, kv4
from test_gpu_kv4 import Setup, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def own_random_numbers(cuda):
    """The same inputs whatever ran before, and none taken from what runs behind."""
    with torch.random.fork_rng(devices=[cuda]):
        torch.manual_seed(2024)
        yield


def busy(stream):
    """Some 50 ms of work on the stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


@pytest.mark.parametrize("new", [1, 70])
def test_default_stream_given_inside_another(cuda, new):
    """The default stream's handle is 0; given, it is the one that is used."""
    r = np.random.default_rng(30)
    st = Setup(cuda, r, [new], [3000], 2, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(1))
    q = torch.randn(st.T, 8, 128, device=cuda).bfloat16()
    k = torch.randn(st.T, 2, 128, device=cuda).bfloat16()
    kv4.append(None, k, k, st.cache, *st.args)
    want = kv4.attend(q, st.cache, *st.args)
    k_want, v_want = kv4.gather(st.cache, *st.args, tokens=st.T, head_dim=128)
    out, qo, ko, vo = (torch.zeros_like(x) for x in (want, q, k_want, v_want))
    ws = abi.kv4_workspace(st.T, 8, 2, 128, 1, device=cuda)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    default = torch.cuda.default_stream()
    busy(side)
    with torch.cuda.stream(side):
        abi.kronq_kv4_append(q, k, k, st.cache, *st.args, q_out=qo, stream=default)
        abi.kronq_kv4_gather(st.cache, *st.args, ko, vo, stream=default)
        abi.kronq_kv4_attention(q, st.cache, *st.args, out=out, ws=ws, stream=default)
    default.synchronize()
    waiting = not side.query()
    got = [x.to("cpu") for x in (out, qo, ko, vo)] if waiting else []
    torch.cuda.synchronize()
    assert waiting                                 # (else nothing was shown)
    for x, w in zip(got, (want, q, k_want, v_want)):
        assert torch.equal(x, w.cpu())


@pytest.mark.parametrize("new", [1, 70])
def test_allocations_belong_to_the_given_stream(cuda, new):
    """While a call waits on a stream of its own, memory is allocated, written and freed on the
    current one: nothing of the call's is among it."""
    r = np.random.default_rng(31)
    st = Setup(cuda, r, [new], [20000], 2, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(1))
    q = torch.randn(st.T, 8, 128, device=cuda).bfloat16()
    k = torch.randn(st.T, 2, 128, device=cuda).bfloat16()
    want_q = kv4.append(q, k, k, st.cache, *st.args, rope=kv4.rope_table(20000, 128, device=cuda))
    want = kv4.attend(want_q, st.cache, *st.args)
    rope = kv4.rope_table(20000, 128, device=cuda)
    need = abi.kronq_kv4_attention_workspace_size(st.T, 8, 2, 128, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        busy(side)
        got_q = abi.kronq_kv4_append(q, k, k, st.cache, *st.args, table=rope, stream=side)
        got = abi.kronq_kv4_attention(got_q, st.cache, *st.args, stream=side)
        for n in (need, need, want.numel() * 2, 256):
            torch.full((n,), 127, dtype=torch.uint8, device=cuda)
        torch.cuda.synchronize()
        assert torch.equal(got_q, want_q) and torch.equal(got, want)


@pytest.mark.parametrize("new,heads", [(1, 2), (90, 2), (2, 1)])
@pytest.mark.parametrize("B,first", [(3, 1), (20, 7), (40, 33), (300, 200), (2000, 1200)])
def test_row_starts_that_decrease(cuda, new, heads, B, first):
    """Where q_start goes back, that sequence and the ones behind it, whose rows others may claim, are
    left out: noticed, the ones in front are right, and what an earlier call left in the workspace
    has no part in the result."""
    r = np.random.default_rng(B)
    L, D = 3000, 128
    st = Setup(cuda, r, [new], [L], heads, D, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(5))
    bt = t(np.repeat(st.bt, B, 0), cuda)                  # (all over the same pages)
    T, g = B * new, 4
    q = torch.randn(T, heads * g, D, device=cuda).bfloat16()
    kv = torch.randint(L // 2, L + 1, (B,), generator=torch.Generator(cuda).manual_seed(6), device=cuda,
                       dtype=torch.int32)
    start = torch.arange(B + 1, device=cuda, dtype=torch.int32) * new
    need = abi.kronq_kv4_attention_workspace_size(T, heads * g, heads, D, B)
    ws = torch.empty(need, dtype=torch.uint8, device=cuda)
    good = kv4.attend(q, st.cache, bt, start, kv, ws=ws)
    stale = ws.clone()
    bad = start.clone()
    bad[first + 1:] -= (start[first + 1] - start[first // 2]).item()     # rows from here on a second time
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    outs = []
    for fill in ("stale", 0, 127):
        ws.copy_(stale) if fill == "stale" else ws.fill_(fill)
        info.zero_()
        lse = torch.full((T, heads * g), 5.0, device=cuda)
        out = torch.full_like(q, 5.0)
        kv4.attend(q, st.cache, bt, bad, kv, out=out, lse=lse, ws=ws, info=info)
        assert info.item() == -1
        outs.append((out, lse))
    n = first * new                                       # rows of the sequences in front
    for out, lse in outs:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
        assert (out[n:] == 5).all() and (lse[n:] == 5).all()
    # (fewer sequences are split otherwise: not the same bits)
    seqs = sorted({0, first - 1})
    st.new, st.kv, st.start = [new] * B, kv.tolist(), start.cpu().numpy()
    st.bt = bt.cpu().numpy()
    check_attention(st, q, outs[0][0], D ** -0.5, rows=[0, new // 2, new - 1], seqs=seqs)
    check_attention(st, q, good, D ** -0.5, rows=[0], seqs=seqs)


@pytest.mark.parametrize("heads", [1, 8])
def test_append_and_gather_notice_bad_rows(cuda, heads):
    """q_start that goes back or leaves the tensor's rows is noticed; no token goes to a place that is
    not one of its sequence's new tokens."""
    r = np.random.default_rng(50)
    D, P, B, n = 64, 16, 100, 3
    st = Setup(cuda, r, [n] * B, [40] * B, heads, D, P)
    T = B * n
    k = torch.randn(T, heads, D, device=cuda).bfloat16()
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    kv4.append(None, k, k, st.cache, *st.args, info=info)
    kv4.gather(st.cache, *st.args, tokens=T, head_dim=D, info=info)
    assert info.item() == 0
    back, beyond, before = (st.args[1].clone() for _ in range(3))
    back[60:] -= 50 * n
    beyond[B] = T + 2
    before[0] = -2
    for start in (back, beyond, before):
        st.cache.fill_(255)
        info.zero_()
        kv4.append(None, k, k, st.cache, st.args[0], start, st.args[2], info=info)
        assert info.item() == -1
        # only slots 37 .. 39 of a sequence can be new tokens
        raw = st.cache.cpu().numpy()
        for b in range(B):
            blk = raw[st.bt[b]]
            kc, _, kw, _ = ok.split_block(blk, P, D)
            free = np.ones((3, P), dtype=bool)
            free[2, 5:8] = False
            assert (kw[np.broadcast_to(free[:, None], kw.shape)] == 0xFFFFFFFF).all()
        info.zero_()
        kv4.gather(st.cache, st.args[0], start, st.args[2], tokens=T, head_dim=D, info=info)
        assert info.item() == -1


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("entry", [-2 ** 31, -1, 2 ** 31 - 1])
def test_any_bad_page_number_is_noticed(cuda, new, entry):
    r = np.random.default_rng(51)
    st = Setup(cuda, r, [new], [400], 1, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(7))
    q = torch.randn(st.T, 4, 128, device=cuda).half()
    bt = st.bt.copy()
    bt[0, 2] = entry
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    kv4.attend(q, st.cache, t(bt, cuda), *st.args[1:], info=info)
    assert info.item() == -1
    info.zero_()                                   # nobody sees it: it may be anything
    kv4.attend(q, st.cache, t(bt, cuda), *st.args[1:], window=100, info=info)
    assert info.item() == 0


def test_an_empty_step(cuda):
    """No sequences: nothing to do, and no error."""
    D, cache = 128, kv4.make_cache(3, 16, 2, 128, cuda)
    cache.fill_(9)
    batch = (torch.empty(0, 4, dtype=torch.int32, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda),
             torch.empty(0, dtype=torch.int32, device=cuda))
    k = torch.empty(0, 2, D, dtype=torch.bfloat16, device=cuda)
    q = torch.empty(0, 8, D, dtype=torch.bfloat16, device=cuda)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    assert kv4.append(q, k, k, cache, *batch, rope=kv4.rope_table(8, D, device=cuda), info=info).shape == q.shape
    assert kv4.attend(q, cache, *batch, info=info).shape == q.shape
    assert kv4.gather(cache, *batch, tokens=0, head_dim=D, info=info)[0].shape == k.shape
    assert info.item() == 0 and (cache == 9).all()
    with pytest.raises(abi.KronqError):
        kv4.attend(torch.empty(1, 8, D, dtype=torch.bfloat16, device=cuda), cache, *batch)


@pytest.mark.parametrize("D,rot,inter,signs", [(128, 128, False, False), (128, 64, False, False), (64, 64, False, True),
                                               (256, 128, False, False), (128, 32, True, False)])
@pytest.mark.parametrize("T", [5, 2000])
def test_queries_rotated_in_place(cuda, D, rot, inter, signs, T):
    r = np.random.default_rng(52)
    st = Setup(cuda, r, [T], [T], 2, D, 64)
    q = torch.randn(T, 6, D, device=cuda).bfloat16()
    k = torch.randn(T, 2, D, device=cuda).bfloat16()
    sg = t((1 - 2 * r.integers(0, 2, D)).astype(np.int8), cuda) if signs else None
    more = dict(rope=kv4.rope_table(T, rot, device=cuda), interleaved=inter, signs=sg)
    want = kv4.append(q, k, k, st.cache, *st.args, **more)
    got = q.clone()
    kv4.append(got, k, k, st.cache, *st.args, q_out=got, **more)
    assert torch.equal(got, want)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_over_its_queries(cuda, new, dtype):
    """The output over the queries, contiguous and within a projection's rows; beside them."""
    r = np.random.default_rng(53)
    st = Setup(cuda, r, [new, new], [9000, 500], 2, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(8))
    q = torch.randn(st.T, 8, 128, device=cuda).to(dtype)
    want = kv4.attend(q, st.cache, *st.args)
    got = q.clone()
    kv4.attend(got, st.cache, *st.args, out=got)
    assert torch.equal(got, want)
    wide = torch.randn(st.T, 20, 128, device=cuda).to(dtype)
    keep = wide.clone()
    wide[:, 3:11] = q
    kv4.attend(wide[:, 3:11], st.cache, *st.args, out=wide[:, 11:19])
    assert torch.equal(wide[:, 11:19], want) and torch.equal(wide[:, 3:11], q)
    kv4.attend(wide[:, 3:11], st.cache, *st.args, out=wide[:, 3:11])
    assert torch.equal(wide[:, 3:11], want)
    assert torch.equal(wide[:, :3], keep[:, :3]) and torch.equal(wide[:, 19:], keep[:, 19:])
    for out in (wide[:, 4:12], wide[:, 1:9]):
        with pytest.raises(abi.KronqError):
            kv4.attend(wide[:, 3:11], st.cache, *st.args, out=out)
    with pytest.raises(abi.KronqError):
        kv4.attend(q, st.cache, *st.args, out=want[:, :1].expand(st.T, 8, 128))


def small_call(cuda):
    """Arguments that each call takes as they are."""
    cache = kv4.make_cache(4, 16, 2, 128, cuda)
    cache.zero_()
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device=cuda)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=cuda)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    return q, k, cache, i32(0, 1, 2, 3)[None], i32(0, 3), i32(3)


def test_append_refusals_on_the_device(cuda):
    q, k, cache, bt, qs, kv = small_call(cuda)
    good = dict(q=q, k=k, v=k, cache=cache, block_table=bt, q_start=qs, kv_len=kv)
    rope, signs = torch.zeros(4, 128, device=cuda), torch.ones(128, dtype=torch.int8, device=cuda)
    good.update(rope=rope, signs=signs, positions=torch.zeros(3, dtype=torch.int32, device=cuda),
                info=torch.zeros(1, dtype=torch.int32, device=cuda), q_out=torch.empty_like(q))
    kv4.append(**good)
    for change, what in (
            (dict(k=k.float()), "k must be bfloat16 or float16"), (dict(v=k.half()), "v must be"),
            (dict(q=q.half()), "q must be"), (dict(k=k[0]), "k must have 3 dims"),
            (dict(v=k[:2]), r"v has shape \(2, 2, 128\), expected \(3, heads, 128\)"),
            (dict(v=k[:, :, :64]), "v has shape"), (dict(q=q[:2]), "q has shape"),
            (dict(v=k[:, :1]), "differ in their heads"), (dict(cache=cache[:, :1].contiguous()), "differ in their heads"),
            (dict(v=torch.zeros(3, 128, 2, dtype=k.dtype, device=cuda).transpose(1, 2)), "unit stride"),
            (dict(cache=cache.view(torch.int8)), "contiguous uint8"), (dict(cache=cache[:, :1]), "contiguous uint8"),
            (dict(cache=cache[0]), "contiguous uint8"),
            (dict(cache=cache[:, :, :-1].contiguous()), "does not hold whole tokens"),
            (dict(block_table=bt.long()), "must be int32"), (dict(q_start=qs.long()), "must be int32"),
            (dict(kv_len=kv.long()), "must be int32"), (dict(block_table=bt[0]), "block_table has 2 dims"),
            (dict(q_start=qs[:1]), "q_start 1 entries"), (dict(kv_len=qs), "kv_len 2"),
            (dict(block_table=bt.repeat(1, 2)[:, ::2]), "unit stride"),
            (dict(block_table=bt.expand(2, 4), q_start=qs.new_zeros(3), kv_len=qs), "rows overlap"),
            (dict(rope=rope.double()), "table must hold"), (dict(rope=rope[0]), "table must have 2 dims"),
            (dict(rope=rope[:, ::2]), "table must hold"), (dict(signs=signs[:64]), "signs must hold 128"),
            (dict(signs=signs.int()), "signs must hold"), (dict(positions=good["positions"][:2]), "positions must hold 3"),
            (dict(positions=good["positions"].long()), "positions must hold"),
            (dict(info=torch.zeros(2, dtype=torch.int32, device=cuda)), "info must hold 1"),
            (dict(q_out=torch.empty_like(q)[:, :, :64]), "q_out must be"), (dict(q_out=q.half()), "q_out must be"),
            (dict(q=None), "q and q_out go together"),
            (dict(k=k.cpu()), "k must be a CUDA tensor"), (dict(v=k.cpu()), "v is on cpu"), (dict(q=q.cpu()), "q is on cpu"),
            (dict(cache=cache.cpu()), "cache is on cpu"), (dict(block_table=bt.cpu()), "block_table is on cpu"),
            (dict(q_start=qs.cpu()), "q_start is on cpu"), (dict(kv_len=kv.cpu()), "kv_len is on cpu"),
            (dict(rope=rope.cpu()), "table is on cpu"), (dict(signs=signs.cpu()), "signs is on cpu"),
            (dict(q_out=torch.empty_like(q).cpu()), "q_out is on cpu")):
        with pytest.raises(ValueError, match=what):
            kv4.append(**{**good, **change})
    for change in (dict(rope=rope[:, :8].contiguous()), dict(rope=torch.zeros(4, 144, device=cuda)),
                   dict(rope=rope[:0]), dict(cache=torch.zeros(4, 2, 24 * 136, dtype=torch.uint8, device=cuda))):
        with pytest.raises(abi.KronqError):
            kv4.append(**{**good, **change})


def test_attention_refusals_on_the_device(cuda):
    q, k, cache, bt, qs, kv = small_call(cuda)
    good = dict(q=q, cache=cache, block_table=bt, q_start=qs, kv_len=kv, out=torch.empty_like(q),
                lse=torch.zeros(3, 4, device=cuda), info=torch.zeros(1, dtype=torch.int32, device=cuda),
                ws=abi.kv4_workspace(3, 4, 2, 128, 1, device=cuda))
    kv4.attend(**good)
    for change, what in (
            (dict(q=q.float()), "q must be bfloat16 or float16"), (dict(q=q[0]), "q must have 3 dims"),
            (dict(q=torch.zeros(3, 128, 4, dtype=q.dtype, device=cuda).transpose(1, 2)), "unit stride"),
            (dict(q=q[:, :, :64]), "does not hold whole tokens|out has shape"),
            (dict(out=q.half()), "out must be"), (dict(out=q[:2]), "out has shape"), (dict(out=q[:, :2]), "out has shape"),
            (dict(out=torch.zeros(3, 4, 256, dtype=q.dtype, device=cuda)[:, :, ::2]), "unit stride"),
            (dict(lse=torch.zeros(3, 3, device=cuda)), "lse has shape"), (dict(lse=torch.zeros(12, device=cuda)), "lse has shape"),
            (dict(lse=torch.zeros(3, 4, dtype=torch.float64, device=cuda)), "lse must hold"),
            (dict(lse=torch.zeros(3, 8, device=cuda)[:, ::2]), "lse must hold"),
            (dict(info=torch.zeros(1, device=cuda)), "info must hold"), (dict(window=-1), "must not be negative"),
            (dict(sinks=-1), "must not be negative"), (dict(ws=good["ws"][::2]), "ws must be contiguous"),
            (dict(q_start=qs[:1]), "q_start 1 entries"), (dict(kv_len=kv.long()), "must be int32"),
            (dict(cache=cache[:, :, :-1].contiguous()), "does not hold whole tokens"),
            (dict(out=q.cpu()), "out is on cpu"), (dict(lse=good["lse"].cpu()), "lse is on cpu"),
            (dict(ws=good["ws"].cpu()), "ws is on cpu"), (dict(info=good["info"].cpu()), "info is on cpu")):
        with pytest.raises(ValueError, match=what):
            kv4.attend(**{**good, **change})
    for change in (dict(q=q[:, :3], out=None, lse=None), dict(window=4, causal=False), dict(scale=float("nan")),
                   dict(ws=good["ws"][:256])):
        with pytest.raises(abi.KronqError):
            kv4.attend(**{**good, **change})


def test_gather_refusals_on_the_device(cuda):
    _, k, cache, bt, qs, kv = small_call(cuda)
    kv4.gather(cache, bt, qs, kv, 3, 128)
    for args, what in (((cache, bt, qs, kv, -1, 128), "must not be negative"), ((cache, bt, qs, kv, 3, 0), "must not be negative"),
                       ((cache, bt, qs, kv, 3, 100), "does not hold whole tokens"), ((cache[0], bt, qs, kv, 3, 128), "3 dims"),
                       ((cache, bt, qs, kv, 3, 128, torch.float64), "must be bfloat16, float16 or float32")):
        with pytest.raises(ValueError, match=what):
            kv4.gather(*args)
    for ko, vo, what in ((k, k.half(), "v_out must be"), (k, k[:2], "v_out must be"), (k.transpose(0, 1), k, "contiguous"),
                         (k[:, :1].contiguous(), k[:, :1].contiguous(), "differ in their heads"), (k.cpu(), k, "CUDA tensor"),
                         (k, k.cpu(), "v_out is on cpu")):
        with pytest.raises(ValueError, match=what):
            abi.kronq_kv4_gather(cache, bt, qs, kv, ko, vo)


@pytest.mark.parametrize("new", [2, 70])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_padding_in_front_and_behind(cuda, new, dtype):
    """Rows in front of the first sequence and behind the last, full of NaN: left as they were, and of no
    effect; the first sequence has no new tokens."""
    r = np.random.default_rng(54)
    st = Setup(cuda, r, [0, new, new], [100, 900, 300], 2, 128, 64)
    st.fill_fast(torch.Generator(cuda).manual_seed(9))
    a, b = 5, 5 + st.T
    T = b + 7
    start = st.args[1] + 5
    wide = torch.full((T, 12, 128), float("nan"), device=cuda).to(dtype)
    wide[a:b] = torch.randn(st.T, 12, 128, device=cuda).to(dtype)
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    rope = kv4.rope_table(900, 64, device=cuda)
    info = torch.zeros(1, dtype=torch.int32, device=cuda)
    before = st.cache.clone()
    want_q = kv4.append(q[a:b], k[a:b], v[a:b], st.cache, *st.args, rope=rope)
    want_cache = st.cache.clone()
    want = kv4.attend(want_q, st.cache, *st.args)
    want_k, want_v = kv4.gather(st.cache, *st.args, tokens=st.T, head_dim=128, dtype=dtype)
    st.cache.copy_(before)
    args = (st.args[0], start, st.args[2])
    q_out = torch.full((T, 8, 128), 3.0, dtype=dtype, device=cuda)
    kv4.append(q, k, v, st.cache, *args, rope=rope, q_out=q_out, info=info)
    assert torch.equal(st.cache, want_cache) and torch.equal(q_out[a:b], want_q)
    assert (q_out[:a] == 3).all() and (q_out[b:] == 3).all()
    out = torch.full((T, 8, 128), 3.0, dtype=dtype, device=cuda)
    lse = torch.full((T, 8), 3.0, device=cuda)
    q_out[:a], q_out[b:] = float("nan"), float("nan")
    kv4.attend(q_out, st.cache, *args, out=out, lse=lse, info=info)
    ko, vo = (torch.full((T, 2, 128), 3.0, dtype=dtype, device=cuda) for _ in range(2))
    abi.kronq_kv4_gather(st.cache, *args, ko, vo, info)
    assert info.item() == 0
    for got, w in ((out, want), (ko, want_k), (vo, want_v)):
        assert torch.equal(got[a:b], w) and (got[:a] == 3).all() and (got[b:] == 3).all()
    assert (lse[:a] == 3).all() and (lse[b:] == 3).all() and (lse[a:b] != 3).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_beyond_32_bits(cuda, D):
    """A cache of 5 GB, used at both of its ends: byte offsets pass 2^32."""
    r = np.random.default_rng(55)
    P, heads = 256, 4
    block = abi.kronq_kv4_block_bytes(P, D)
    pages = (5 << 30) // (heads * block)
    assert (pages - 3) * heads * block > 1 << 32
    big = kv4.make_cache(pages, P, heads, D, cuda)
    for new in (1, 40):
        small = Setup(cuda, r, [new, new], [700, 600], heads, D, P)
        small.fill_fast(torch.Generator(cuda).manual_seed(10))
        ids = torch.tensor([pages - 1, 0, pages - 2, pages // 2, 1, pages - 3, pages - 4, 2], device=cuda)
        assert small.pages <= len(ids)
        big[ids[:small.pages]] = small.cache
        bt = torch.where(small.args[0] >= 0, ids[small.args[0].clamp_min(0).long()], -1).int()
        k = torch.randn(small.T, heads, D, device=cuda).bfloat16()
        q = torch.randn(small.T, heads * 4, D, device=cuda).bfloat16()
        outs = []
        for cache, table in ((small.cache, small.args[0]), (big, bt)):
            kv4.append(None, k, k.flip(0), cache, table, *small.args[1:])
            outs.append((kv4.attend(q, cache, table, *small.args[1:]),
                         *kv4.gather(cache, table, *small.args[1:], tokens=small.T, head_dim=D)))
        assert all(torch.equal(x, y) for x, y in zip(*outs))
