"""Refusals of the 4-bit cache's entry points, on the host: through the C ABI
(nothing is launched) and through the binding's own checks."""

import ctypes
import pathlib

import pytest
import torch

from post_quantization_02_b200 import abi, build, kv4


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


P = ctypes.c_void_p(4096)   # never dereferenced: refused before any launch


def _append(L, **kw):
    a = dict(q=P, qt=512, qh=128, k=P, kt=512, kh=128, v=P, vt=512, vh=128, dtype=0, T=4, q_heads=4, q_out=P,
             table=P, rows=16, rot=128, inter=0, pos=None, signs=None, cache=P, pages=8, page=16, heads=2, D=128,
             bt=P, ld=4, mp=4, qs=P, kv=P, B=2)
    a.update(kw)
    return L.kronq_kv4_append(a["q"], a["qt"], a["qh"], a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["dtype"],
                              a["T"], a["q_heads"], a["q_out"], a["table"], a["rows"], a["rot"], a["inter"], a["pos"],
                              a["signs"], a["cache"], a["pages"], a["page"], a["heads"], a["D"], a["bt"], a["ld"],
                              a["mp"], a["qs"], a["kv"], a["B"], None, None)


def _attend(L, **kw):
    a = dict(q=P, qt=512, qh=128, dtype=0, T=4, q_heads=4, cache=P, pages=8, page=16, heads=2, D=128, bt=P, ld=4, mp=4,
             qs=P, kv=P, B=2, scale=0.1, causal=1, window=0, sinks=0, out=P, ot=512, oh=128, lse=None, ws=P, n=None)
    a.update(kw)
    n = L.kronq_kv4_attention_workspace_size(4, 4, 2, 128, 2) if a["n"] is None else a["n"]
    return L.kronq_kv4_attention(a["q"], a["qt"], a["qh"], a["dtype"], a["T"], a["q_heads"], a["cache"], a["pages"],
                                 a["page"], a["heads"], a["D"], a["bt"], a["ld"], a["mp"], a["qs"], a["kv"], a["B"],
                                 ctypes.c_float(a["scale"]), a["causal"], a["window"], a["sinks"], a["out"], a["ot"],
                                 a["oh"], a["lse"], None, a["ws"], n, None)


def test_block_bytes(L):
    assert L.kronq_kv4_block_bytes(64, 128) == 64 * 136
    assert L.kronq_kv4_block_bytes(24, 128) == 0 and L.kronq_kv4_block_bytes(512, 128) == 0
    assert L.kronq_kv4_block_bytes(64, 96) == 0


SHARED = [
    (dict(D=96), -2), (dict(page=48), -2), (dict(page=8), -2), (dict(page=512), -2), (dict(cache=None), -1),
    (dict(cache=ctypes.c_void_p(4104)), -1), (dict(pages=0), -1), (dict(pages=1 << 31), -1), (dict(heads=0), -1),
    (dict(B=0), -1), (dict(qs=None), -1), (dict(kv=None), -1), (dict(bt=None), -1), (dict(ld=3), -1),
    (dict(mp=-1), -1), (dict(mp=1 << 27, ld=1 << 27), -2), (dict(dtype=2), -2), (dict(dtype=9), -2), (dict(T=-1), -1),
    (dict(qs=ctypes.c_void_p(4098)), -1),
]


@pytest.mark.parametrize("kw,code", SHARED)
def test_refusals_of_both(L, kw, code):
    assert _append(L, **kw) == code
    assert _attend(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(q_out=None), -1),
    (dict(q_out=ctypes.c_void_p(4104)), -1), (dict(k=ctypes.c_void_p(4097)), -1), (dict(kt=-512), -1),
    (dict(rot=8), -1), (dict(rot=144), -1), (dict(rot=-16), -1), (dict(table=None), -1), (dict(rows=0), -1),
    (dict(table=ctypes.c_void_p(4100)), -1), (dict(pos=ctypes.c_void_p(4098)), -1), (dict(q_heads=-1), -1),
    (dict(T=0), 0),
])
def test_append_refusals(L, kw, code):
    assert _append(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(out=ctypes.c_void_p(4100)), -1), (dict(ot=510), -1),
    (dict(q_heads=5), -1), (dict(q_heads=0), -1), (dict(window=-1), -1), (dict(sinks=-1), -1),
    (dict(window=4, causal=0), -1), (dict(scale=float("nan")), -1), (dict(ws=None), -6), (dict(n=1000), -6),
    (dict(ws=ctypes.c_void_p(4112)), -6), (dict(T=0), 0),
])
def test_attention_refusals(L, kw, code):
    assert _attend(L, **kw) == code


def test_workspace_sizes(L):
    f = L.kronq_kv4_attention_workspace_size
    assert f(4, 4, 2, 128, 2) > 0
    assert f(4, 5, 2, 128, 2) == 0 and f(4, 4, 2, 96, 2) == 0 and f(4, 4, 2, 128, 0) == 0 and f(-1, 4, 2, 128, 2) == 0


def test_binding_refusals(L):
    """Types, shapes and devices are refused before the library is called."""
    with pytest.raises(ValueError):
        kv4.make_cache(4, 48, 2, 128, device="cpu")
    cache = kv4.make_cache(4, 16, 2, 128, device="cpu")
    assert cache.shape == (4, 2, 16 * 136)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    bt, qs, kv = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.tensor(
        [3], dtype=torch.int32)
    good = dict(q=q, k=k, v=k, cache=cache, block_table=bt, q_start=qs, kv_len=kv)
    for change in (dict(), dict(k=k.float()), dict(v=k.half()), dict(q=q.half()), dict(v=k[:, :1]), dict(k=k[:2]),
                   dict(block_table=bt.long()), dict(q_start=qs[:1]), dict(kv_len=qs), dict(cache=cache[:, :1]),
                   dict(cache=cache.view(torch.int8)), dict(cache=cache[:, :, :-1]), dict(k=k.transpose(1, 2)),
                   dict(block_table=bt.expand(2, 4), q_start=torch.zeros(3, dtype=torch.int32), kv_len=qs),
                   dict(rope=torch.zeros(4, 128, dtype=torch.float64)), dict(signs=torch.ones(64, dtype=torch.int8)),
                   dict(positions=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):      # the unchanged call: these tensors are not on a GPU
            kv4.append(**{**good, **change})
    good = dict(q=q, cache=cache, block_table=bt, q_start=qs, kv_len=kv, ws=torch.empty(256, dtype=torch.uint8))
    for change in (dict(), dict(q=q.float()), dict(out=q.half()), dict(out=q[:2]), dict(lse=torch.zeros(3, 3)),
                   dict(lse=torch.zeros(3, 4, dtype=torch.float64)), dict(q=q[:, :, :64])):
        with pytest.raises(ValueError):
            kv4.attend(**{**good, **change})
    with pytest.raises(ValueError):
        kv4.gather(cache, bt, qs, kv, 3, 128)


class _Recorder:
    """Stands for the compiled binding: notes the stream that is current at each call."""

    def __init__(self):
        self.current, self.seen = [], []

    def context(self, stream):
        import contextlib

        @contextlib.contextmanager
        def entered():
            self.current.append(stream)
            yield
            self.current.pop()
        return entered()

    def __getattr__(self, name):
        if name not in ("append", "gather", "attention", "gather_new"):
            raise AttributeError(name)

        def call(*args):
            # no argument is a stream's handle: 0 is the default stream's, not "none"
            self.seen.append((name, self.current[-1] if self.current else None, args))
        return call


def test_calls_run_and_allocate_on_the_given_stream(monkeypatch):
    """The stream of a call is current while its outputs and workspace are allocated and its
    kernels launched: what is allocated on another stream may be handed out again while they run.
    The default stream, whose handle is 0, counts as given."""
    rec = _Recorder()
    monkeypatch.setattr(abi, "_kv4_calls", lambda: rec)
    monkeypatch.setattr(torch.cuda, "stream", rec.context)

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    x = torch.zeros(1)
    for s in (None, Stream(0), Stream(77)):
        rec.seen.clear()
        abi.kronq_kv4_append(x, x, x, x, x, x, x, stream=s)
        abi.kronq_kv4_gather(x, x, x, x, x, x, stream=s)
        abi.kronq_kv4_attention(x, x, x, x, x, stream=s)
        kv4.append(x, x, x, x, x, x, x, stream=s)
        kv4.gather(x, x, x, x, 1, 64, stream=s)
        kv4.attend(x, x, x, x, x, stream=s)
        assert len(rec.seen) == 6
        for name, current, args in rec.seen:
            assert current is s, name
            assert not any(type(a) is int and a == 77 for a in args), name


def test_nothing_to_do(L):
    """No sequences and no tokens (a step in which nothing is scheduled) is no error; tokens of no
    sequence's are."""
    empty = dict(T=0, B=0, kv=None, bt=None)
    assert _append(L, **empty) == 0 and _attend(L, **empty) == 0 and _attend(L, **empty, ws=None, n=0) == 0
    assert _append(L, **empty, k=None, v=None, q=None, q_out=None) == 0
    assert L.kronq_kv4_gather(None, None, 0, 0, P, 8, 16, 2, 128, None, 4, 4, P, None, 0, None, None) == 0
    for some in (dict(B=0), dict(B=0, kv=None, bt=None)):
        assert _append(L, **some) == -1 and _attend(L, **some) == -1
    assert _append(L, T=0, B=-1) == -1 and _attend(L, T=0, B=-1) == -1


def at(elements):
    """An address so many 16-bit elements behind P."""
    return ctypes.c_void_p(P.value + 2 * elements)


@pytest.mark.parametrize("kw,code", [
    # rows of the output that share memory
    (dict(ot=0), -1), (dict(oh=0), -1), (dict(ot=256), -1), (dict(oh=64), -1), (dict(ot=508), -1),
    (dict(ot=128, oh=508), -1), (dict(T=1, ot=0), -6), (dict(ot=128, oh=512), -6), (dict(ot=1024, oh=256), -6),
    # the output over the queries: only as they lie
    (dict(out=at(0)), -6), (dict(out=at(128)), -1), (dict(out=at(512)), -1), (dict(out=at(4 * 512)), -6),
    (dict(q=at(512), out=at(0)), -1), (dict(out=at(0), ot=1024), -1),
    # ... or beside them in the same buffer
    (dict(qt=1024, ot=1024, out=at(512)), -6), (dict(qt=1024, ot=1024, out=at(1024 + 512)), -6),
    (dict(qt=1024, ot=1024, out=at(508)), -1), (dict(qt=1024, ot=1024, out=at(516)), -1),
    (dict(qt=1024, ot=1024, out=at(1024)), -1),
])
def test_outputs_that_overlap(L, kw, code):
    """-6: the arguments are taken (the workspace, which is too small here, is looked at last)."""
    assert _attend(L, **{**dict(n=0, out=at(1 << 20)), **kw}) == code


@pytest.mark.parametrize("kw", [dict(q_out=at(8)), dict(q_out=at(512)), dict(q=at(512)), dict(qt=1024),
                                dict(qh=256, qt=1024), dict(k=at(16)), dict(k=at(2047)), dict(v=at(1000))])
def test_rotated_queries_that_overlap_inputs(L, kw):
    far = dict(q=P, q_out=P, k=at(1 << 20), v=at(1 << 21))
    assert _append(L, **{**far, **kw}) == -1


def test_binding_is_rebuilt_for_another_torch(L, monkeypatch, tmp_path):
    """The binding is compiled against torch's headers: with another torch installed it is stale."""
    calls = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        calls.append(cmd)
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_bytes(b"")
        return Done()

    src = tmp_path / "kv4_torch.cpp"
    src.write_text("")
    monkeypatch.setattr(build, "BINDING", tmp_path / "_kv4.so")
    monkeypatch.setattr(build, "BINDING_SRC", src)
    monkeypatch.setattr(build, "INCLUDE", tmp_path)
    monkeypatch.setattr(build, "OBJ", tmp_path / "_build")
    monkeypatch.setattr(build.subprocess, "run", run)
    build._build_binding()
    build._build_binding()
    assert len(calls) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build._build_binding()
    build._build_binding()
    assert len(calls) == 2
