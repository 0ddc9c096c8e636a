"""The join of partials that are not numbers: a split that attended something and whose sum is NaN (a
CTA that gave up waiting, a query that is not finite) makes the head's output and lse NaN; it is not
taken for a head that attended nothing, whose output is 0 and lse -inf."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_kv_cache_gb300 as K
    K.load()
    return K


def join(K, acc, m, l, sink=None):
    units, ns, G, D = acc.shape
    lse = torch.full((units * G,), 7.0, device="cuda")
    out = K.split_combine(acc, m, l, units * G, units, sink, lse=lse)
    torch.cuda.synchronize()
    return out.view(units, G, D).cpu().numpy(), lse.view(units, G).cpu().numpy()


def partials(D, ns, units=2, G=3, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return r(units, ns, G, D), r(units, ns, G), r(units, ns, G).abs() + 0.5


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ns", [1, 3, 32])
@pytest.mark.parametrize("sink", [False, True])
def test_a_nan_sum_gives_nan(K, D, ns, sink):
    acc, m, l = partials(D, ns)
    s = torch.zeros(6, device="cuda") if sink else None
    o0, l0 = join(K, acc, m, l, s)
    k = ns - 1
    l[0, k, 1] = float("nan")
    o, e = join(K, acc, m, l, s)
    assert np.isnan(o[0, 1]).all() and np.isnan(e[0, 1])
    keep = np.ones((2, 3), bool)
    keep[0, 1] = False
    assert np.array_equal(o[keep], o0[keep]) and np.array_equal(e[keep], l0[keep])
    assert np.isfinite(o[keep]).all() and np.isfinite(e[keep]).all()


def test_a_nan_sum_without_weight_gives_nan(K):
    # its exponent is so far below the others' that its weight is 0
    acc, m, l = partials(128, 4)
    m[1, 2, 0], l[1, 2, 0] = -3.0e38, float("nan")
    o, e = join(K, acc, m, l)
    assert np.isnan(o[1, 0]).all() and np.isnan(e[1, 0])
    assert np.isfinite(o[0]).all() and np.isfinite(o[1, 1:]).all()


def test_an_infinite_maximum_gives_nan(K):
    # what the staged prefill publishes for a CTA that gave up
    acc, m, l = partials(256, 5)
    acc[1, 3, 2], m[1, 3, 2], l[1, 3, 2] = float("nan"), float("inf"), float("nan")
    o, e = join(K, acc, m, l)
    assert np.isnan(o[1, 2]).all() and np.isnan(e[1, 2])
    assert np.isfinite(o[0]).all() and np.isfinite(o[1, :2]).all()


def test_empty_splits_stay_empty(K):
    acc, m, l = partials(64, 4)
    o0, e0 = join(K, acc[:, :2].contiguous(), m[:, :2].contiguous(), l[:, :2].contiguous())
    acc[:, 2:], m[:, 2:], l[:, 2:] = float("nan"), float("-inf"), 0.0
    o, e = join(K, acc, m, l)
    assert np.array_equal(o, o0) and np.array_equal(e, e0)
    m[:], l[:] = float("-inf"), 0.0
    o, e = join(K, acc, m, l)
    assert not o.any() and np.isneginf(e).all()
