"""Draft trees (kvq_attend_tree) under a softcap and with a per-channel K scale
at head_dim 128, over every type and both sides of 64 query rows: scores within
the cap's polynomial, beyond it and far in its saturation.

Tolerances as in test_gpu_tree; a logit is off by 2^-16 of sum |q k| more (256
fp32 additions of partial sums up to that), which larger queries show."""
import dataclasses

import numpy as np
import pytest

import score_ref as ref
import step_ref
from test_gpu_tree import run

pytestmark = pytest.mark.gpu

INT8, FP8, INT4 = ref.INT8, ref.FP8, ref.INT4
ROW, TENSOR, CHANNEL = ref.ROW, ref.TENSOR, ref.CHANNEL


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def check(c: ref.Cache, got, parents, nodes, sink=None):
    out, lse = got
    r_out, r_lse, absv, f16, size = step_ref.attend_tree(c, parents, nodes, sink)
    ds = (2.0 ** -11 if c.case.km == CHANNEL else 2.0 ** -16) * size + 2.0 ** -15
    empty = r_lse == -np.inf
    if lse is not None:
        assert (lse[empty] == -np.inf).all() and np.isfinite(lse[~empty]).all()
        # (a per-channel scale's query comes in two parts when an lse is asked for)
        e = np.abs(lse[~empty] - r_lse[~empty]) - ((2.0 ** -16 * size + 2.0 ** -15)[~empty]
                                                   + 2.0 ** -20 * (1 + np.abs(r_lse[~empty])))
        assert e.size == 0 or e.max() <= 0, f"lse off by {e.max():.2e} more than its bound"
    assert (out[empty] == 0).all() and np.isfinite(out).all()
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    worst = (np.abs(out - r_out) / tol).max()
    assert worst <= 1.0, f"output {worst:.2f} times its bound"


KINDS = {
    "int8 row d128": ref.Case(hq=8, hkv=2),
    "int8 row d256": ref.Case(d=256, hq=6, hkv=1, bs=32),
    "int8 channel d128": ref.Case(km=CHANNEL, vm=TENSOR, hq=16, hkv=2),
    "int8 channel d256": ref.Case(km=CHANNEL, vm=ROW, d=256, hq=4, hkv=1),
    "int8 tensor d256": ref.Case(km=TENSOR, vm=TENSOR, d=256, hq=4, hkv=1),
    "fp8 row d128": ref.Case(dtype=FP8, hq=4, hkv=1),
    "fp8 row d256": ref.Case(dtype=FP8, d=256, hq=4, hkv=1),
    "fp8 channel d128": ref.Case(dtype=FP8, km=CHANNEL, vm=CHANNEL, hq=8, hkv=2),
    "fp8 channel d256": ref.Case(dtype=FP8, km=CHANNEL, vm=CHANNEL, d=256, hq=4, hkv=1),
    "int4 row d128": ref.Case(dtype=INT4, hq=8, hkv=2),
    "int4 row d256": ref.Case(dtype=INT4, d=256, hq=6, hkv=1, bs=32),
    "int4 channel d128": ref.Case(dtype=INT4, km=CHANNEL, vm=ROW, hq=8, hkv=2),
    "int4 channel d256": ref.Case(dtype=INT4, km=CHANNEL, vm=CHANNEL, d=256, hq=6, hkv=1),
}


def trees(case, T, seed):
    cache = ref.Cache(dataclasses.replace(case, c=T, seed=seed, lens=(400 + T, T + 5)))
    parents = step_ref.random_parents(np.random.default_rng(seed), 2, T)
    return cache, parents, np.array([T, max(1, T - 2)])


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("T", [5, 11, 30])
@pytest.mark.parametrize("cap,amp", [(0.0, 1.0), (2.0, 1.0), (2.0, 8.0), (50.0, 1.0), (50.0, 8.0), (50.0, 40.0)])
def test_caps_and_channel_scales(kvq, name, T, cap, amp):
    cache, parents, nodes = trees(dataclasses.replace(KINDS[name], softcap=cap, amp=amp), T, T)
    check(cache, run(kvq, cache, parents, nodes), parents, nodes)
    out, _ = run(kvq, cache, parents, nodes, lse=False)
    check(cache, (out, None), parents, nodes)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 channel d128", "int4 channel d256", "fp8 row d256"])
@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_caps_with_windows_and_sinks(kvq, name, cap):
    case = dataclasses.replace(KINDS[name], softcap=cap, amp=4.0, window=70)
    cache, parents, nodes = trees(case, 21, 3)
    sink = np.linspace(-1, 2, case.hq)
    check(cache, run(kvq, cache, parents, nodes, sink), parents, nodes, sink)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 channel d128", "int4 row d256", "fp8 row d128", "int4 channel d256"])
@pytest.mark.parametrize("T", [2, 3, 4])
def test_few_rows_beside_a_long_table(kvq, name, T):
    """A table for more than 65,536 keys takes 9 to 16 rows to the tiles."""
    case = dataclasses.replace(KINDS[name], c=T, seed=T, lens=(500 + T, T + 70), hkv=1, hq=4)
    cache = ref.Cache(case, width=40000 // KINDS[name].bs)
    parents = step_ref.random_parents(np.random.default_rng(T), 2, T)
    nodes = np.array([T, T - 1])
    check(cache, run(kvq, cache, parents, nodes), parents, nodes)
    check(cache, (run(kvq, cache, parents, nodes, lse=False)[0], None), parents, nodes)
