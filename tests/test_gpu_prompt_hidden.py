"""Packed prompts (kvq_attend_prompt) whose K and V rows hold infinities or NaN:
a token's result has them where it sees them and nowhere else, to the bit.

A weight of 0 times a finite number leaves a sum as it is, so the results are
those of the same call with zeros in place of the bad elements, except for the
channels in which a token sees one: these are not finite."""
import numpy as np
import pytest
import torch

from test_gpu_prompt import check, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def sees_bad(v, cu, window):
    """[N, Hkv, D]: whether a token sees an element that is not finite."""
    bad, got, bounds = ~torch.isfinite(v.float()), torch.zeros(v.shape, dtype=torch.bool, device="cuda"), cu.tolist()
    for s0, s1 in zip(bounds, bounds[1:]):
        n = bad[s0:s1].int().cumsum(0)
        if window and s1 - s0 > window:
            n[window:] -= n[:-window].clone()
        got[s0:s1] = n > 0
    return got


def compare(kvq, x, bad_v, window, **kw):
    """One call over V with bad elements against one with zeros there."""
    q, k, v, cu = x
    G = q.shape[1] // k.shape[1]
    spoilt = torch.where(torch.isfinite(bad_v), v, bad_v)
    clean = torch.where(torch.isfinite(bad_v), v, torch.zeros_like(v))
    want = run(kvq, q, k, clean, cu, window=window, **kw)
    got = run(kvq, q, k, spoilt, cu, window=window, **kw)
    there = sees_bad(spoilt, cu, window).repeat_interleave(G, 1)
    assert there.any() and not there.all()
    assert torch.equal(got[0][~there], want[0][~there])
    assert not torch.isfinite(got[0][there].float()).any()
    assert torch.equal(got[1], want[1])
    return clean, want


def sprinkle(shape, at, what, seed=0, whole=False):
    """Zeros but for `what` in the rows `at`, in some channels of some heads or in all."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    for i in at:
        t[i] = torch.where(torch.rand(shape[1:], generator=g, device="cuda") < (2.0 if whole else 0.05), what, 0.0)
        t[i, -1, i % shape[2]] = what
    return t


SHAPES = [(4, 1, 64), (8, 2, 128), (6, 1, 256), (3, 1, 128), (7, 1, 64), (10, 2, 256), (2, 2, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 20, 128, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_reach_the_tokens_that_see_them(kvq, hq, hkv, d, window, bad):
    lens = (333, 1, 140, 257)
    x = inputs(lens, hq, hkv, d, seed=window + hq)
    at = [126, 127, 128, 129, 250, 332, 334, 400, 474 + 255]
    clean, want = compare(kvq, x, sprinkle(x[2].shape, at, bad, seed=window), window)
    if bad != bad:
        check(x[0], x[1], clean, x[3], want, window=window)
    compare(kvq, x, sprinkle(x[2].shape, [40, 474 + 130], bad, whole=True), window)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 64), (32, 8, 128), (24, 4, 256), (24, 8, 128)])
@pytest.mark.parametrize("window", [0, 500])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_bad_values_in_long_prompts(kvq, hq, hkv, d, window, cap):
    """Units of two row tiles, many of them a CTA."""
    x = inputs((2500, 1100), hq, hkv, d, seed=d)
    at = [700, 1279, 1280, 1281, 2499, 2500, 3000]
    compare(kvq, x, sprinkle(x[2].shape, at, float("nan")), window, cap=cap)


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 50, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_keys_reach_the_tokens_that_see_them(kvq, hq, hkv, d, window, bad):
    q, k, v, cu = inputs((300, 140), hq, hkv, d, seed=window)
    want = run(kvq, q, k, v, cu, window=window)
    spoilt = sprinkle(k.shape, [127, 128, 200, 310], bad, whole=True)
    got = run(kvq, q, torch.where(torch.isfinite(spoilt), k, spoilt), v, cu, window=window)
    there = sees_bad(spoilt, cu, window).repeat_interleave(hq // hkv, 1)
    assert there.any() and not there.all()
    assert torch.equal(got[0][~there], want[0][~there])
    assert torch.equal(got[1][~there[..., 0]], want[1][~there[..., 0]])


def test_bad_values_and_the_junk_behind_a_sequence(kvq):
    """Rows behind the last sequence hold NaN, the last rows of it too."""
    for d in (64, 128, 256):
        x = inputs((130, 40, 1), 8, 2, d, before=5, behind=70)
        v = sprinkle(x[2].shape, [5 + 129, 5 + 130 + 39], float("nan"), whole=True)
        zero = torch.zeros_like(x[2])
        zero[5:176] = x[2][5:176]
        want = run(kvq, *x[:2], torch.where(torch.isfinite(v), zero, torch.zeros_like(zero)), x[3])
        got = run(kvq, *x[:2], torch.where(torch.isfinite(v), x[2], v), x[3])
        there = torch.zeros(x[0].shape[0], dtype=torch.bool, device="cuda")
        there[5 + 129], there[5 + 130 + 39] = True, True
        assert torch.equal(got[0][~there], want[0][~there]) and not torch.isfinite(got[0][there].float()).any()


def test_many_short_sequences_with_bad_values(kvq):
    r = np.random.default_rng(5)
    lens = tuple(int(n) for n in r.integers(0, 40, 700))
    x = inputs(lens, 8, 2, 128, seed=4)
    at = [int(i) for i in r.choice(sum(lens), 60, replace=False)]
    compare(kvq, x, sprinkle(x[2].shape, at, float("nan")), 0)
    compare(kvq, x, sprinkle(x[2].shape, at, float("inf")), 6)
