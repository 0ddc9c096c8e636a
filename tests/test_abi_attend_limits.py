"""paged_prefill's workspace without a GPU: a size that suits every batch of a serving loop."""
import itertools
import os

import pytest


@pytest.fixture(scope="module")
def K():
    import int8_kv_cache_gb300 as K
    if not os.path.exists(K.library_path()):
        from int8_kv_cache_gb300 import build
        build.build()
    K.load()
    return K


def test_a_workspace_for_every_batch(K):
    """What the header names suits every T and B, and the need does not grow with them."""
    f = K.paged_prefill_workspace_bytes
    for D, n in itertools.product((64, 128, 256), (2, 152, 1024)):
        most = f(256, 1, 8, 8, D, 4096, n)
        assert most == n * 2 * (128 if D == 256 else 256) * (D + 2) * 4
        sizes = {f(T, B, Hq, Hkv, D, cap, n) for T, B, cap in itertools.product((1, 63, 191, 192, 4096, 1 << 20), (1, 2, 64, 4096),
                 (1, 128, 4096, (1 << 31) - 512)) for Hq, Hkv in ((8, 8), (32, 8), (16, 1))}
        assert max(sizes) == most
    assert f(256, 4, 8, 8, 128, 4096, 8) < f(256, 1, 8, 8, 128, 4096, 8)
