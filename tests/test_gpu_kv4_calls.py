"""The 4-bit key/value cache's calls on the GPU: streams, refusals, batches that contradict
themselves.  (What they compute: test_gpu_kv4.py.)"""

import numpy as np
import pytest
import torch

from post_quantization_02_b200 import abi, kv4
from test_gpu_kv4 import Setup

pytestmark = pytest.mark.gpu


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
