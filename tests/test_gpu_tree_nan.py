"""Draft trees (kvq_attend_tree) that hold NaN or infinities where a node sees
them: its result is NaN, not what is left without them, on every kernel; the
other nodes' results stay within their bounds."""
import dataclasses

import numpy as np
import pytest

import score_ref as ref
import step_ref
from test_gpu_masked import CASES, gpu_cache
from test_gpu_tree import run
from test_gpu_tree_hidden import expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def check_others(c, got, parents, nodes, spoilt):
    """spoilt [B, T, Hq]: the rows that are NaN."""
    out, lse = got
    r_out, r_lse, absv, f16, size = expected(c, parents, nodes)
    ds = ((2.0 ** -11 if c.case.km == ref.CHANNEL else 0.0) + c.case.d * 2.0 ** -24) * size + 2.0 ** -15
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    assert np.isnan(out[spoilt]).all() and np.isnan(lse[spoilt]).all()
    assert (np.abs(out - r_out) <= tol)[~spoilt].all()
    assert (np.abs(lse - r_lse) <= ds + 2.0 ** -20 * (1 + np.abs(r_lse)))[~spoilt].all()


KINDS = [("int8 row d128", 2), ("int8 row d128", 5), ("int8 row d128", 40), ("int8 row d256 g6", 3), ("int8 row d256 g6", 16),
         ("fp8 row", 20), ("int8 channel d64", 3), ("int8 channel d64", 9), ("int4 channel d256", 4), ("int4 channel d256", 13),
         ("int4 row", 4), ("int4 group", 5), ("fp8 group v", 3), ("latent d256", 6), ("latent d576", 2), ("latent d576", 6)]


def trees(name, T, lens=(900, 0), **kw):
    """(Several CTAs share the first sequence; the other is its nodes alone.)"""
    cache = ref.Cache(dataclasses.replace(CASES[name], c=T, seed=T, lens=tuple(L + T for L in lens), **kw))
    parents = step_ref.random_parents(np.random.default_rng(T), len(lens), T)
    return cache, parents, np.full(len(lens), T)


@pytest.mark.parametrize("name,T", KINDS)
@pytest.mark.parametrize("window", [0, 1])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_query_that_is_not_finite(kvq, name, T, window, bad):
    cache, parents, nodes = trees(name, T, window=window)
    spoilt = np.zeros(cache.q.shape[:3], bool)
    spoilt[0, T - 1, 0] = spoilt[1, T // 2, -1] = True
    kept = cache.q.copy()
    cache.q[spoilt] = bad
    for flags in (0, kvq.DECODE_NO_TCGEN05):
        got = run(kvq, cache, parents, nodes, flags=flags)
        q, cache.q = cache.q, kept
        check_others(cache, got, parents, nodes, spoilt)
        cache.q = q


@pytest.mark.parametrize("name,T", [k for k in KINDS if "channel" not in k[0]])
def test_a_node_that_is_not_finite_reaches_its_descendants(kvq, name, T):
    cache, parents, nodes = trees(name, T)
    at = T // 2  # (a node in the middle: itself and those below it)
    spoilt = np.zeros(cache.q.shape[:3], bool)
    for b in range(len(nodes)):
        for i, chain in enumerate(step_ref.chains(parents[b], T)):
            spoilt[b, i] = at in chain
    g = gpu_cache(kvq, cache)
    case = cache.case
    for b, L in enumerate(case.lens):
        pos = L - T + at
        page, row = int(cache.table[b, pos // case.bs]), pos % case.bs
        if case.km in (ref.ROW, ref.GROUP):
            g.k_scale[page, :, row] = np.nan
        if case.vm in (ref.ROW, ref.GROUP) and not case.latent:
            g.v_scale[page, :, row] = np.nan
    for flags in (0, kvq.DECODE_NO_TCGEN05):
        got = run(kvq, cache, parents, nodes, flags=flags, gcache=g)
        if case.km not in (ref.ROW, ref.GROUP):  # the value alone: the lse is that of the scores
            assert np.isnan(got[0][spoilt]).all()
            got[1][spoilt] = np.nan
        check_others(cache, got, parents, nodes, spoilt)
