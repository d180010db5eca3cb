"""Sizes at which kvd_attend_paged_prefix's lengths meet 32 bits (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from decode_attention_kv_gb300 import _build, kvd
    _build.build()
    return kvd.load()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("BS", [1, 5, 24, 128])
def test_prefixes_of_two_to_the_31_tokens(lib, BS, dtype):
    """A length is rounded up to whole key tiles of at most 128 in 32 bits: tables that hold more
    than 2^31 - 128 tokens are refused (lengths above that counted as no prefix)."""
    most = (2 ** 31 - 128) // BS
    f = lib.kvd_attend_paged_prefix_workspace_bytes
    assert f(1, 1, 1, 1, BS, most, 1, 64, dtype) > 0
    assert f(1, 1, 1, 1, BS, most + 1, 1, 64, dtype) == 0
    assert "pcols*BS" in lib.kvd_last_error().decode()
    assert lib.kvd_attend_paged_prefix(None, None, None, None, None, None, None, None, None, None,
                                       None, 1, 1, 1, 1, 4, BS, most + 1, 1, 64, 0.1, dtype, None,
                                       0, None, None) == 2
