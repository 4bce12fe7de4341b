"""The by-parts frequencies where the ramp ends past the last pair (no GPU)."""
import math

import pytest

import exact_attention_14_gb300 as ea


@pytest.fixture(scope="module", autouse=True)
def lib():
    from exact_attention_14_gb300 import _build
    _build.build()
    return ea.load()


@pytest.mark.parametrize("rot,base,length,slow", [
    (128, 10000.0, 131072, 1.0), (64, 10000.0, 65536, 1.0), (128, 10000.0, 65536, 1.0), (6, 10000.0, 4096, 1.0),
    (64, 10000.0, 131072, 1.0), (32, 10000.0, 8192, 0.25), (4, 1000.0, 1 << 20, 1.0), (128, 10000.0, 1 << 30, 0.001),
    (128, 500000.0, 8192, 1.0), (128, 10000.0, 4096, 1.0), (250, 1e6, 32768, 1.0)])
@pytest.mark.parametrize("fast", [32.0, 2.0])
@pytest.mark.parametrize("factor", [1.0, 4.0, 32.0])
def test_the_ramp(rot, base, length, slow, fast, factor):
    """The share of f / factor in each pair, from the pair that turns a number of times: told by
    counting turns, base^(-2 i / rot) * length / (2 pi), not by a logarithm."""
    got, _ = ea.attn_rope_frequencies(rot, base, scaling="by_parts", factor=factor, original_len=length,
                                      beta_fast=fast, beta_slow=slow)
    pairs = rot // 2
    plain = [base ** (-2.0 * i / rot) for i in range(pairs)]

    def turns(i):                       # of pair i, were there as many
        return base ** (-2.0 * i / rot) * length / (2 * math.pi)
    # the ramp's ends, outwards: the last pair that turns at least `fast` times and the first one
    # that turns at most `slow` times, within 0 and rot - 1
    first = max([i for i in range(rot) if turns(i) >= fast], default=0)
    last = min([i for i in range(rot) if turns(i) <= slow], default=rot - 1)
    for i, (g, f) in enumerate(zip(got, plain)):
        r = min(max((i - first) / max(last - first, 1e-3), 0.0), 1.0)
        assert math.isclose(g, f / factor * r + f * (1 - r), rel_tol=1e-12)
        if turns(i) >= fast:
            assert math.isclose(g, f, rel_tol=1e-12)
        if factor > 1 and math.isclose(g, f / factor, rel_tol=1e-12) and i != last:
            assert turns(i) <= slow     # divided in full: slow, or where the ramp's end was rounded to
