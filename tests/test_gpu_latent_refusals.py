"""What the latent calls refuse, and that they refuse before anything runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def z(*shape, dtype=BF, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def attend_args(R=128, P=64):
    return dict(q_latent=z(2, 1, 4, R), q_rope=z(2, 1, 4, P), latent_cache=z(6, 16, 1, R),
                rope_cache=z(6, 16, 1, P), block_tables=z(2, 3, dtype=I32),
                seq_lens=z(3, dtype=I32), scale=0.1)


@pytest.mark.parametrize("change, error", [
    (lambda: dict(q_latent=z(2, 1, 4, 128, dtype=F32)), TypeError),            # types differ
    (lambda: dict(q_rope=z(2, 1, 4, 32)), ValueError),                         # rows do not fit the cache
    (lambda: dict(q_latent=z(2, 4, 128)), ValueError),                         # no token axis
    (lambda: dict(q_latent=z(2, 1, 4, 256)[..., ::2]), ValueError),            # not contiguous
    (lambda: dict(q_latent=z(2, 1, 4, 128, device="cpu")), ValueError),
    (lambda: dict(latent_cache=z(6, 16, 128)), ValueError),
    (lambda: dict(latent_cache=z(6, 16, 2, 128)), ValueError),                 # two heads
    (lambda: dict(rope_cache=z(6, 8, 1, 64)), ValueError),                     # other pages
    (lambda: dict(block_tables=z(2, 3, dtype=torch.int64)), TypeError),
    (lambda: dict(block_tables=z(3, 3, dtype=I32)), ValueError),
    (lambda: dict(seq_lens=z(2, dtype=I32)), ValueError),
    (lambda: dict(seq_offset=z(3, dtype=I32)), ValueError),
    (lambda: dict(out=z(2, 1, 4, 64)), ValueError),
    (lambda: dict(lse=z(2, 1, 4)), TypeError),
    (lambda: dict(workspace=z(16, dtype=torch.uint8, device="cpu")), ValueError),
    (lambda: dict(dev_status=z(1, dtype=torch.int64)), ValueError),
    (lambda: dict(scale=None), TypeError),
    (lambda: dict(q_latent=None), TypeError),
    (lambda: dict(latent_cache=z(6, 16, 1, 128, dtype=torch.float16)), TypeError),
])
def test_attend_latent(kvd, change, error):
    with pytest.raises(error):
        kvd.attend_latent(**{**attend_args(), **change()})


def test_attend_latent_library_errors(kvd):
    with pytest.raises(kvd.KvdError) as e:
        kvd.attend_latent(**attend_args(R=192))
    assert e.value.status == "KVD_ERR_UNSUPPORTED" and "192" in str(e.value)
    with pytest.raises(kvd.KvdError) as e:
        kvd.attend_latent(**attend_args(), workspace=z(256, dtype=torch.uint8))
    assert e.value.status == "KVD_ERR_WORKSPACE"
    args = attend_args()
    args["q_rope"] = z(2 * 4 * 64 + 1)[1:].view(2, 1, 4, 64)           # 2 bytes off 16
    with pytest.raises(kvd.KvdError) as e:
        kvd.attend_latent(**args)
    assert e.value.status == "KVD_ERR_INVALID_ARG"
    out = kvd.attend_latent(**attend_args())                            # lengths of zero
    assert bool((out == 0).all())


@pytest.mark.parametrize("change, error", [
    (lambda: dict(latent_new=z(5, 64)), ValueError),
    (lambda: dict(rope_new=z(4, 64)), ValueError),
    (lambda: dict(latent_new=z(5, 128, dtype=F32)), TypeError),
    (lambda: dict(new_lens=z(2, dtype=I32)), ValueError),
    (lambda: dict(pos=z(2, dtype=torch.int64)), TypeError),
    (lambda: dict(block_tables=z(3, dtype=I32)), ValueError),
    (lambda: dict(latent_new=z(128)), ValueError),
])
def test_append_latent(kvd, change, error):
    args = dict(latent_cache=z(6, 16, 1, 128), rope_cache=z(6, 16, 1, 64),
                block_tables=z(2, 3, dtype=I32), seq_offset=None, latent_new=z(5, 128),
                rope_new=z(5, 64), new_lens=z(3, dtype=I32), pos=z(2, dtype=I32))
    with pytest.raises(error):
        kvd.append_latent(**{**args, **change()})


@pytest.mark.parametrize("change, error", [
    (lambda: dict(q=z(4, 192)), ValueError),
    (lambda: dict(kv=z(4, 3, 256)), ValueError),                               # other heads
    (lambda: dict(kv=z(4, 2, 100)), ValueError),                               # no room for values
    (lambda: dict(k_rope=z(3, 64)), ValueError),
    (lambda: dict(k_rope=z(4, 64, dtype=F32)), TypeError),
    (lambda: dict(q_lens=z(3, dtype=I32)), ValueError),
    (lambda: dict(out=z(4, 2, 64)), ValueError),
])
def test_attend_expanded(kvd, change, error):
    args = dict(q=z(4, 2, 192), kv=z(4, 2, 256), k_rope=z(4, 64), q_lens=z(2, dtype=I32),
                k_lens=z(2, dtype=I32))
    with pytest.raises(error):
        kvd.attend_expanded(**{**args, **change()})


def test_attend_expanded_library_errors(kvd):
    with pytest.raises(kvd.KvdError) as e:
        kvd.attend_expanded(z(4, 2, 160), z(4, 2, 224), z(4, 64), z(2, dtype=I32), z(2, dtype=I32))
    assert e.value.status == "KVD_ERR_UNSUPPORTED"


@pytest.mark.parametrize("change, error", [
    (lambda: dict(target_probs=z(2, 50, dtype=F32)), ValueError),
    (lambda: dict(draft_probs=z(2, 3, 49, dtype=F32)), ValueError),
    (lambda: dict(draft_probs=z(2, 3, 50)), TypeError),
    (lambda: dict(draft_probs=None), TypeError),
    (lambda: dict(draft_tokens=z(2, 3, dtype=torch.int64)), TypeError),
    (lambda: dict(u_accept=z(3, 2, dtype=F32)), ValueError),
    (lambda: dict(u_sample=z(2, dtype=torch.float64)), TypeError),
    (lambda: dict(num_drafts=z(1, dtype=I32)), ValueError),
    (lambda: dict(tokens=z(2, 3, dtype=I32)), ValueError),
])
def test_verify_drafts(kvd, change, error):
    args = dict(target_probs=z(2, 4, 50, dtype=F32), draft_probs=z(2, 3, 50, dtype=F32),
                draft_tokens=z(2, 3, dtype=I32), u_accept=z(2, 3, dtype=F32),
                u_sample=z(2, dtype=F32))
    with pytest.raises(error):
        kvd.verify_drafts(**{**args, **change()})


def test_empty_batches(kvd):
    """No sequences: nothing runs, outputs have no rows."""
    a = attend_args()
    a.update(q_latent=z(0, 1, 4, 128), q_rope=z(0, 1, 4, 64), block_tables=z(0, 3, dtype=I32),
             seq_lens=z(1, dtype=I32))
    assert kvd.attend_latent(**a).shape == (0, 1, 4, 128)
    kvd.append_latent(z(6, 16, 1, 128), z(6, 16, 1, 64), z(0, 3, dtype=I32), None, z(0, 128),
                      z(0, 64), z(1, dtype=I32), z(0, dtype=I32))
    t, n = kvd.verify_drafts(z(0, 4, 50), z(0, 3, 50), z(0, 3, dtype=I32), z(0, 3, dtype=F32),
                             z(0, dtype=F32))
    assert t.shape == (0, 4) and n.shape == (0,)
