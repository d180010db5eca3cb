"""The latent calls on several streams and from several host threads at once:
every result is that of the call alone."""
import threading

import pytest
import torch

import latent_ref as ref
from test_gpu_expanded import Packed
from test_gpu_verify import draws

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def calls(kvd, dtype):
    """Each call over inputs of its own, as a function without arguments that returns tensors."""
    c = ref.LatentCase([700, 3, 90], 2, 12, 256, 32, dtype, seed=1)
    e = Packed([300, 17, 129], [300, 80, 129], 3, 128, 64, dtype, seed=2)
    p, q, x, u, us = draws(9, 3, 4001, dtype, seed=3)
    new = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 30], dtype=torch.int32, device="cuda")
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    cn, rn = (torch.randn(3, w, device="cuda").to(dtype) for w in (128, 64))

    def attend():
        lse = torch.empty(c.ql.shape[:3], device="cuda")
        return kvd.attend_latent(c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, c.scale,
                                 seq_offset=c.seq_offset, lse=lse), lse

    def expanded():
        lse = torch.zeros(e.q.shape[:2], device="cuda")
        return kvd.attend_expanded(e.q, e.kv, e.kr, e.ql, e.kl, e.scale, lse=lse,
                                   out=torch.zeros(e.q.shape[0], 3, 64, dtype=dtype,
                                                   device="cuda")), lse

    def append():
        latent, rope = (torch.zeros(6, 16, 1, w, dtype=dtype, device="cuda") for w in (128, 64))
        kvd.append_latent(latent, rope, table, None, cn, rn, new, pos)
        return latent, rope

    return [attend, expanded, append, lambda: kvd.verify_drafts(p, q, x, u, us)]


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_two_streams(kvd, dtype):
    """The same call on two streams at once, each call in turn; workspaces and
    outputs are allocated inside."""
    for f in calls(kvd, dtype):
        want = f()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for _ in range(10):
            for s in streams:
                with torch.cuda.stream(s):
                    got.append(f())
        torch.cuda.synchronize()
        assert all(same(g, want) for g in got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_host_threads(kvd, dtype):
    """All calls from four threads, a stream each, in other orders."""
    fs = calls(kvd, dtype)
    want = [f() for f in fs]
    torch.cuda.synchronize()
    got = [[] for _ in range(4)]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for k in range(40):
                j = (i + k * (2 * (i & 1) + 1)) % len(fs)
                got[i].append((j, fs[j]()))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g in got:
        assert len(g) == 40
        assert all(same(r, want[j]) for j, r in g)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_two_graphs_that_allocate_inside(kvd, dtype):
    """Two captures of all calls, with outputs and workspaces from the graphs' own
    memory, replayed on two streams at once."""
    fs = calls(kvd, dtype)
    want = [f() for f in fs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([f() for f in fs])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for results in got:
        assert all(same(r, w) for r, w in zip(results, want))
