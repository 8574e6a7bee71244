"""The bound of kv_accuracy.py on the CPU: outputs with the kernels' roundings are within it, wrong ones are not: zeros, a page left
out or taken twice, a part of the keys with a wrong weight, a query with one term where two are kept."""
import pytest
import torch

from compressed_sparse_long_append_b200.layer import DenseShape
from kv_accuracy import attend64, bound, head_ratios, ratios

BF, F32 = torch.bfloat16, torch.float32


def _data(D, HQ, HK, t, L, window=0, mul=1.0, seed=0, d_rope=64):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(BF)   # noqa: E731
    shape = DenseShape(D=D, HQ=HQ, HK=HK, d_rope=d_rope, window=window)
    return shape, r(t, HQ, D) * mul, r(L, HK, D), r(L, HK, D), torch.randn(HQ, generator=g)


@pytest.mark.parametrize("D,HQ,HK,t,L,window", [(128, 4, 1, 1, 70001, 0), (64, 8, 4, 3, 20011, 0), (128, 4, 4, 2, 17000, 0),
                                                (64, 4, 1, 2, 30000, 3000), (128, 2, 2, 2, 900, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("terms", [1, 2])
def test_right_outputs_pass_and_wrong_ones_fail(D, HQ, HK, t, L, window, dtype, terms):
    shape, q, k, v, sink = _data(D, HQ, HK, t, L, window)
    args = (q, k, v, L - t, shape, False, sink, None)
    o, spread = attend64(*args)
    most = bound(dtype, terms, spread, HQ * D)
    assert most < 0.01
    got = attend64(*args, terms=terms, weights=BF)[0].to(dtype)
    assert bool((ratios(got, o) <= most).all()), (ratios(got, o), most)
    assert bool((ratios(torch.zeros_like(got), o) > 0.99).all())
    # the last whole page that the first row sees, out or twice: as a mask over tokens with one log-weight each
    page = (L - t) // 128 - 1

    def without(lo, hi, weight):
        """The output with tokens lo..hi-1 counted `weight` times."""
        part = attend64(q, k, v, L - t, DenseShape(D=D, HQ=HQ, HK=HK, d_rope=64, window=window), False, sink, None)[0]
        vz = v.clone()
        vz[lo:hi] = 0
        rest = attend64(q, k, vz, L - t, shape, False, sink, None)[0]
        ones = torch.zeros_like(v)
        ones[lo:hi] = 1
        share = attend64(q, k, ones, L - t, shape, False, sink, None)[0]
        return (rest + weight * (part - rest)) / (1 + (weight - 1) * share)

    assert torch.allclose(without(0, L, 1.0), o)
    for weight in (0.0, 2.0):
        bad = without(128 * page, 128 * page + 128, weight).to(dtype)
        assert bool((ratios(bad, o) > most).all()), (weight, ratios(bad, o), most)
    # an eighth of the keys that are seen with a weight off by a fifth: a maximum or a join that went wrong
    lo = L - t - (window or L - t) // 8
    bad = without(lo, L - t, 1.2).to(dtype)
    assert bool((ratios(bad, o) > most).all()), (ratios(bad, o), most)


@pytest.mark.parametrize("D,HQ,HK,t", [(128, 32, 8, 1), (64, 64, 8, 1), (64, 8, 4, 8)])
def test_a_sharper_query_needs_both_terms(D, HQ, HK, t):
    """Scores of a spread of 2 over 20000 keys (some hundreds of them count): one term of the query is beyond the bound of two."""
    for seed in range(4):
        shape, q, k, v, sink = _data(D, HQ, HK, t, 20000, mul=2.0, seed=seed, d_rope=D)
        args = (q, k, v, 20000 - t, shape, False, sink, None)
        o, spread = attend64(*args)
        assert 1.8 < spread < 3.2
        most = bound(F32, 2, spread, t * HQ * D)
        two, one = (head_ratios(attend64(*args, terms=n, weights=BF)[0].float(), o).median() for n in (2, 1))
        assert two <= most < one, (two, one, most)
