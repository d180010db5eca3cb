"""Host refusals of the serving step's entry points, and the rotary frequencies (no
GPU needed)."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from decode_attention_kv_gb300 import _build, kvd
    _build.build()
    return kvd.load()


def P(x):
    return None if x is None else ctypes.c_void_p(x * 4096)


ODD = ctypes.c_void_p(4096 + 2)


def test_plan_pages_validates(lib):
    def call(bt=P(1), held=P(1), free=P(1), lens=P(1), slots=P(1), Q=2, N=4, BS=16, cols=4, F=8):
        return lib.kvd_plan_pages(bt, held, free, P(1), P(1), lens, None, P(1), slots, P(1), Q, N,
                                  BS, cols, F, None, None)
    for bad in (dict(bt=None), dict(held=None), dict(free=None), dict(lens=None), dict(slots=None),
                dict(Q=-1), dict(N=-1), dict(BS=0), dict(cols=0), dict(F=-1), dict(bt=ODD)):
        assert call(**bad) == 1, bad
    assert call(Q=(1 << 20) + 1) == 2 and call(N=(1 << 30) + 1) == 2


def test_rotate_validates(lib):
    def call(x=P(1), w=None, f=P(1), pos=P(1), out=P(1), N=4, H=2, D=128, Dr=64, dt=0):
        return lib.kvd_rotate(x, w, f, pos, out, N, H, D, Dr, 0, 1.0, 1e-6, dt, None, None)
    for bad in (dict(x=None), dict(f=None), dict(pos=None), dict(out=None), dict(N=-1), dict(H=0),
                dict(dt=3), dict(x=ODD), dict(w=ODD), dict(f=ctypes.c_void_p(4100))):
        assert call(**bad) == 1, bad
    for bad in (dict(D=96), dict(Dr=24), dict(Dr=144), dict(Dr=-16), dict(H=70000)):
        assert call(**bad) == 2, bad
    assert call(N=0, x=None) == 0


def test_rotate_append_validates(lib):
    def call(x=P(1), slots=P(1), kc=P(1), N=4, Hq=4, Hkv=2, NB=8, BS=16, D=128, Dr=128, dt=0):
        return lib.kvd_rotate_append_paged(x, None, None, P(1), P(1), slots, P(1), kc, P(1), N, Hq,
                                           Hkv, NB, BS, D, Dr, 0, 1.0, 1e-6, dt, None, None)
    for bad in (dict(x=None), dict(slots=None), dict(kc=None), dict(Hq=0), dict(Hkv=0), dict(NB=0),
                dict(BS=0), dict(N=-1), dict(dt=7), dict(kc=ODD)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=32, Dr=32), dict(Dr=8), dict(NB=1 << 28, BS=16)):
        assert call(**bad) == 2, bad
    assert call(N=0, x=None) == 0


def test_attend_paged_prefix_validates(lib):
    f = lib.kvd_attend_paged_prefix_workspace_bytes

    def call(q=P(1), pt=P(1), Q=4, G=2, Hq=8, Hkv=2, NB=64, BS=16, pcols=8, cols=4, D=128, dt=0,
             ws=P(1), wsb=None):
        if wsb is None:
            wsb = f(Q, G, Hq, Hkv, BS, pcols, cols, D, dt)
        return lib.kvd_attend_paged_prefix(q, P(1), P(1), pt, P(1), P(1), P(1), P(1), None, P(1),
                                           None, Q, G, Hq, Hkv, NB, BS, pcols, cols, D, 0.1, dt, ws,
                                           wsb, None, None)
    for bad in (dict(q=None), dict(pt=None), dict(q=ODD), dict(NB=0), dict(ws=ODD)):
        assert call(**bad) == 1, bad
    for bad in (dict(Q=-1), dict(G=-1), dict(Hq=6, Hkv=4), dict(BS=0), dict(pcols=0), dict(cols=0),
                dict(dt=2)):
        assert call(**bad, wsb=0) == 1, bad
        b = dict(Q=4, G=2, Hq=8, Hkv=2, BS=16, pcols=8, cols=4, D=128, dt=0) | bad
        assert f(*(b[k] for k in ("Q", "G", "Hq", "Hkv", "BS", "pcols", "cols", "D", "dt"))) == 0
    for bad in (dict(D=96), dict(G=2000), dict(pcols=1 << 28), dict(cols=1 << 28),
                dict(Q=1 << 26)):
        assert call(**bad, wsb=0) == 2, bad
    assert call(NB=1 << 28) == 2
    assert call(ws=None) == 3
    need = f(4, 2, 8, 2, 16, 8, 4, 128, 0)
    assert need > 0 and call(wsb=need - 1) == 3 and str(need) in lib.kvd_last_error().decode()
    assert call(Q=0, q=None, ws=None, wsb=0) == 0
    assert f(4, 0, 8, 2, 16, 1, 4, 128, 0) > 0


def test_sampling_validates(lib):
    def sample(l=P(1), u=P(1), t=P(1), R=2, V=100, dt=0):
        return lib.kvd_sample(l, None, None, None, None, u, t, R, V, dt, None, None)

    def probs(l=P(1), out=P(1), R=2, V=100, dt=0, pt=1):
        return lib.kvd_filter_probs(l, None, None, None, None, out, R, V, dt, pt, None, None)
    for bad in (dict(l=None), dict(u=None), dict(t=None), dict(R=-1), dict(V=0), dict(dt=2),
                dict(u=ODD), dict(l=ctypes.c_void_p(4097))):
        assert sample(**bad) == 1, bad
    for bad in (dict(l=None), dict(out=None), dict(R=-1), dict(V=0), dict(dt=2), dict(pt=5),
                dict(out=ODD)):
        assert probs(**bad) == 1, bad
    assert sample(V=(1 << 20) + 1) == 2 and probs(V=(1 << 20) + 1) == 2
    assert sample(R=0, l=None) == 0 and probs(R=0, l=None, out=None) == 0


def test_rotary_freqs(lib):
    from decode_attention_kv_gb300 import kvd
    i = torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-2 * i / 64)
    got = kvd.rotary_freqs(64, device="cpu")
    assert torch.allclose(got, plain, rtol=1e-14, atol=0)
    assert torch.allclose(kvd.rotary_freqs(64, scaling="linear", factor=4.0, device="cpu"),
                          plain / 4, rtol=1e-14, atol=0)
    # a larger base leaves the fastest frequency and divides the slowest by the factor
    based = kvd.rotary_freqs(64, scaling="base", factor=8.0, device="cpu")
    assert float(based[0]) == 1.0 and math.isclose(float(based[-1]), float(plain[-1]) / 8, rel_tol=1e-12)
    parts = kvd.rotary_freqs(64, scaling="parts", factor=4.0, trained=2048, fast=32, slow=1,
                             device="cpu")
    turns = 2048 * plain / (2 * math.pi)
    assert torch.allclose(parts[turns > 32], plain[turns > 32], rtol=1e-14, atol=0)
    assert torch.allclose(parts[turns < 1], plain[turns < 1] / 4, rtol=1e-14, atol=0)
    mid = (turns >= 1) & (turns <= 32)
    keep = (turns[mid] - 1) / 31
    assert bool(mid.any()) and torch.allclose(
        parts[mid], plain[mid] * (keep + (1 - keep) / 4), rtol=1e-13, atol=0)


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0),
                                 dict(base=math.nan), dict(base=math.inf),
                                 dict(scaling="linear", factor=0.0),
                                 dict(scaling="base", factor=math.nan),
                                 dict(scaling="base", factor=2.0, rotary_dim=2),
                                 dict(scaling="parts", factor=2.0, fast=1.0, slow=1.0),
                                 dict(scaling="parts", factor=2.0, trained=0.0)])
def test_rotary_freqs_refuses(lib, bad):
    from decode_attention_kv_gb300 import kvd
    with pytest.raises(kvd.KvdError):
        kvd.rotary_freqs(**({"rotary_dim": 64} | bad), device="cpu")


def test_rotary_freqs_refuses_a_name(lib):
    from decode_attention_kv_gb300 import kvd
    with pytest.raises(ValueError):
        kvd.rotary_freqs(64, scaling="log", device="cpu")


def test_binding_refuses_before_the_library(lib):
    """Tensors off the GPU, wrong shapes and types raise; nothing is launched."""
    from decode_attention_kv_gb300 import kvd
    z = torch.zeros
    i = torch.int32
    with pytest.raises(ValueError):
        kvd.plan_pages(z(2, 3, dtype=i), z(2, dtype=i), z(4, dtype=i), z(1, dtype=i), z(2, dtype=i),
                       z(3, dtype=i), 16, 4)
    with pytest.raises(ValueError):
        kvd.rotate(z(2, 3, 64), z(2, dtype=i), z(16, dtype=torch.float64))
    with pytest.raises(ValueError):
        kvd.rotate_append_paged(z(2, 4, 64), z(2, 16, 1, 64), z(2, 16, 1, 64), z(2, dtype=i),
                                z(2, dtype=i), z(16, dtype=torch.float64))
    with pytest.raises(ValueError):
        kvd.attend_paged_prefix(z(2, 4, 64), z(2, 16, 1, 64), z(2, 16, 1, 64), z(1, 1, dtype=i),
                                z(1, dtype=i), z(2, dtype=i), z(2, 1, dtype=i), z(3, dtype=i))
    with pytest.raises(ValueError):
        kvd.sample(z(2, 8), z(2))
    with pytest.raises(ValueError):
        kvd.filter_probs(z(2, 8))
    with pytest.raises(TypeError):
        kvd.sample(None, z(2))
