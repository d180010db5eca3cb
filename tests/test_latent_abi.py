"""Host refusals of the latent-cache entry points (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from decode_attention_kv_gb300 import _build, kvd
    _build.build()
    return kvd.load()


def P(x):
    return None if x is None else ctypes.c_void_p(x * 4096)


def test_workspace(lib):
    f = lib.kvd_attend_latent_workspace_bytes
    assert f(1, 1, 16, 128, 8, 512, 64, 0) > 0
    assert f(64, 4, 32, 64, 100, 512, 64, 0) > 0
    assert f(0, 1, 16, 128, 8, 512, 64, 0) > 0
    for bad in ((1, 0, 16, 128, 8, 512, 64, 0), (1, 1, 0, 128, 8, 512, 64, 0),
                (1, 1, 16, 128, 8, 500, 64, 0), (1, 1, 16, 128, 8, 512, 32, 0),
                (1, 1, 16, 128, 8, 512, 64, 9), (70000, 1, 1, 1, 1, 128, 64, 0),
                (1, 70000, 1, 1, 1, 128, 64, 0), (-1, 1, 16, 128, 8, 512, 64, 0),
                (1, 1, 16, 1 << 20, 1 << 20, 512, 64, 0)):
        assert f(*bad) == 0, bad


def _attend(lib, q=1, out=1, Q=2, T=1, H=16, NB=8, BS=64, cols=4, R=512, Pr=64, dt=0, ws=1, wsb=None):
    if wsb is None:
        wsb = lib.kvd_attend_latent_workspace_bytes(Q, T, H, BS, cols, R, Pr, dt)
    return lib.kvd_attend_latent(P(q), P(1), P(1), P(1), P(1), P(1), None, P(out), None, Q, T, H,
                                 NB, BS, cols, R, Pr, 0.1, dt, P(ws), wsb, None, None)


def test_attend_latent_validates(lib):
    assert _attend(lib, q=None) == 1
    assert _attend(lib, out=None) == 1
    assert _attend(lib, NB=0) == 1
    assert _attend(lib, T=0, wsb=0) == 1
    assert _attend(lib, dt=5, wsb=0) == 1
    assert _attend(lib, R=320, wsb=0) == 2
    assert _attend(lib, Pr=128, wsb=0) == 2
    assert _attend(lib, NB=1 << 26, BS=64) == 2
    assert _attend(lib, ws=None) == 3
    need = lib.kvd_attend_latent_workspace_bytes(2, 1, 16, 64, 4, 512, 64, 0)
    assert _attend(lib, wsb=need - 1) == 3
    assert str(need) in lib.kvd_last_error().decode()
    assert _attend(lib, Q=0, q=None, ws=None, wsb=0) == 0
    odd = ctypes.c_void_p(4096 + 8)
    assert lib.kvd_attend_latent(odd, P(1), P(1), P(1), P(1), P(1), None, P(1), None, 2, 1, 16, 8,
                                 64, 4, 512, 64, 0.1, 0, P(1), need, None, None) == 1
    assert lib.kvd_attend_latent(P(1), P(1), P(1), P(1), P(1), P(1), None, P(1), None, 2, 1, 16, 8,
                                 64, 4, 512, 64, 0.1, 0, odd, need, None, None) == 1


def test_append_latent_validates(lib):
    def call(c=1, n=4, Q=2, BS=16, R=512, Pr=64, dt=0):
        return lib.kvd_append_latent(P(c), P(1), P(1), P(1), P(1), None, P(1), P(1), Q, n, 8, BS, 4,
                                     R, Pr, dt, None, None)
    assert call(c=None) == 1
    assert call(R=12) == 1          # rows of whole 16-byte vectors
    assert call(Pr=4) == 1
    assert call(BS=0) == 1
    assert call(dt=3) == 1
    assert call(Q=-1) == 1
    assert call(Q=0, c=None) == 0
    assert call(n=0, c=None) == 0


def test_attend_expanded_validates(lib):
    def call(q=1, Q=2, Nq=8, Nk=8, H=4, Dn=128, Dv=128, Pr=64, dt=0, kv=1):
        return lib.kvd_attend_expanded(P(q), P(kv), P(1), P(1), P(1), P(1), None, Q, Nq, Nk, H, Dn,
                                       Dv, Pr, 0.1, 1, dt, None, None)
    assert call(q=None) == 1
    assert call(kv=None) == 1
    assert call(H=0) == 1
    assert call(dt=2) == 1
    assert call(Dn=96) == 2
    assert call(Dv=192) == 2
    assert call(Pr=32) == 2
    assert call(Q=0, q=None) == 0
    assert call(Nq=0, q=None) == 0


def test_verify_drafts_validates(lib):
    def call(p=1, q=1, x=1, u=1, Q=2, T=3, V=100, dt=0):
        return lib.kvd_verify_drafts(P(p), P(q), P(x), P(u), P(1), None, P(1), P(1), Q, T, V, dt,
                                     None, None)
    assert call(p=None) == 1
    assert call(q=None) == 1
    assert call(x=None) == 1
    assert call(u=None) == 1
    assert call(V=0) == 1
    assert call(T=-1) == 1
    assert call(dt=4) == 1
    assert call(Q=0, p=None) == 0


def test_binding_refuses_before_the_library(lib):
    """Wrong devices, shapes and types raise; nothing is launched."""
    from decode_attention_kv_gb300 import kvd
    z = torch.zeros
    with pytest.raises(ValueError):
        kvd.attend_latent(z(1, 1, 2, 128), z(1, 1, 2, 64), z(2, 16, 1, 128), z(2, 16, 1, 64),
                          z(1, 2, dtype=torch.int32), z(2, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        kvd.attend_expanded(z(4, 2, 192), z(4, 2, 256), z(4, 64), z(2, dtype=torch.int32),
                            z(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvd.append_latent(z(2, 16, 1, 128), z(2, 16, 1, 64), z(1, 2, dtype=torch.int32), None,
                          z(1, 128), z(1, 64), z(2, dtype=torch.int32), z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvd.verify_drafts(z(1, 2, 8), z(1, 1, 8), z(1, 1, dtype=torch.int32), z(1, 1), z(1))
