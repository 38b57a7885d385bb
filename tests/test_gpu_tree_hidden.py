"""Draft trees (kvq_attend_tree) whose nodes' cached rows are far from the
others: a row that a node does not see changes nothing of its result, whatever
it holds.

Tolerances are those of test_gpu_tree, but for the f16 rounding of weights with
a V scale in them: relative to the largest V row that the node itself sees
(step_ref.attend_tree takes the largest of the sequence); and a logit of D
products has D - 1 fp32 additions of partial sums up to sum |q k|, each 2^-24 of
it off, which shows where a latent row's scale makes the logits large too.  (By
2^30 and more nothing of such a row's own softmax is left in fp32: a logit's
rounding passes 2^5.  There only the nodes that do not see it are compared.)"""
import dataclasses

import numpy as np
import pytest

import score_ref as ref
import step_ref
from test_gpu_masked import CASES, gpu_cache
from test_gpu_tree import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def expected(c: ref.Cache, parents, nodes):
    """step_ref.attend_tree with the f16 part of each node by the rows it sees."""
    out, lse, absv, f16, size = step_ref.attend_tree(c, parents, nodes)
    case = c.case
    scale, mode = (c.k_scale, case.km) if case.latent else (c.v_scale, case.vm)
    top = {ref.INT8: 128.0, ref.FP8: 448.0, ref.INT4: 8.0}[case.dtype]
    for b in range(len(case.lens)):
        blk, row = c.rows(b)
        for i, at in enumerate(step_ref.tree_keys(case, parents, nodes, b)):
            for h in range(case.hkv):
                hq = slice(h * case.group, (h + 1) * case.group)
                s = scale[blk[at], h, row[at]] if mode in (ref.ROW, ref.GROUP) else (
                    scale[h] if mode == ref.CHANNEL else scale)
                f16[b, i, hq] = 2.0 ** -10 * absv[b, i, hq] + 2.0 ** -24 * len(at) * top * float(s.max())
    return out, lse, absv, f16, size


def check(c: ref.Cache, got, parents, nodes, only=slice(None)):
    out, lse = got
    r_out, r_lse, absv, f16, size = expected(c, parents, nodes)
    ds = ((2.0 ** -11 if c.case.km == ref.CHANNEL else 0.0) + c.case.d * 2.0 ** -24) * size + 2.0 ** -15
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    out, lse, r_out, r_lse, tol, ds = (x[:, only] for x in (out, lse, r_out, r_lse, tol, ds))
    seen = r_lse > -np.inf
    assert np.isfinite(out).all() and np.isfinite(lse[seen]).all()
    assert (np.abs(lse - r_lse)[seen] <= (ds + 2.0 ** -20 * (1 + np.abs(r_lse)))[seen]).all()
    worst = (np.abs(out - r_out) / tol).max()
    assert worst <= 1.0, f"output {worst:.2f} times its bound"


def enlarge(c: ref.Cache, b, pos, by):
    """The V row (a latent cache's row) at position `pos` of sequence b, `by` times as large."""
    blk, row = c.rows(b)
    (c.k_scale if c.case.latent else c.v_scale)[blk[pos], :, row[pos]] *= np.float32(by)


KINDS = [("int8 row d128", 2), ("int8 row d128", 5), ("int8 row d128", 16), ("int8 row d128", 40),
         ("int8 row d256 g6", 3), ("int8 row d256 g6", 10), ("int8 row d256 g6", 16), ("fp8 row", 3), ("fp8 row", 20),
         ("int4 row", 3), ("int4 row", 33), ("int4 group", 4), ("int4 group", 20), ("fp8 group v", 9),
         ("int8 group k, row v", 7), ("latent d256", 5), ("latent d576", 2), ("latent d576", 6)]


@pytest.mark.parametrize("name,T", KINDS)
@pytest.mark.parametrize("by", [2.0 ** 20, 2.0 ** 30, 2.0 ** 100])
def test_a_large_node_reaches_its_descendants_only(kvq, name, T, by):
    cache, parents, nodes = make(name, T, ragged=False)
    parents[:, -1] = -1  # the last node: a root without children, seen by itself alone
    for b, L in enumerate(cache.case.lens):
        enlarge(cache, b, L - 1, by)
    others = slice(0, T - 1) if cache.case.latent and by > 2.0 ** 20 else slice(None)
    check(cache, run(kvq, cache, parents), parents, nodes, others)


@pytest.mark.parametrize("name,T", [k for k in KINDS if k[1] > 4])
@pytest.mark.parametrize("by", [2.0 ** 12, 2.0 ** 40])
def test_branches_of_different_size(kvq, name, T, by):
    """Two branches under the first node, one of them large: its nodes' results
    are large too, the others' as if it were not there."""
    cache, parents, nodes = make(name, T, ragged=False)
    i = np.arange(T)
    parents[:] = np.maximum(i - 2, 0)
    parents[:, 0] = -1
    for b, L in enumerate(cache.case.lens):
        for n in (1, 3):  # the odd branch
            enlarge(cache, b, L - T + n, by)
    others = slice(0, T, 2) if cache.case.latent and by > 2.0 ** 20 else slice(None)
    check(cache, run(kvq, cache, parents), parents, nodes, others)
    check(cache, run(kvq, cache, parents, flags=kvq.DECODE_NO_TCGEN05), parents, nodes, others)


@pytest.mark.parametrize("name,T", [("int8 row d128", 5), ("int8 row d128", 40), ("int8 row d256 g6", 16), ("fp8 row", 20),
                                    ("int4 row", 9), ("int4 group", 8)])
@pytest.mark.parametrize("cap", [2.0, 50.0])
def test_a_large_node_under_a_cap(kvq, name, T, cap):
    cache, parents, nodes = make(name, T, ragged=False, softcap=cap, amp=4.0)
    parents[:, -1] = -1
    for b, L in enumerate(cache.case.lens):
        enlarge(cache, b, L - 1, 2.0 ** 30)
    check(cache, run(kvq, cache, parents), parents, nodes)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 row d256 g6", "fp8 row", "int4 row", "int4 group"])
@pytest.mark.parametrize("T", [65, 100])
@pytest.mark.parametrize("at", [2, 63, 64])
@pytest.mark.parametrize("by", [2.0 ** 30, 2.0 ** 118])
def test_a_large_node_among_tiles_of_nodes(kvq, name, T, at, by):
    """No prefix, or a short one: no tile is seen whole by all nodes."""
    case = dataclasses.replace(CASES[name], c=T, seed=T, lens=(T, T + 70))
    cache = ref.Cache(case)
    parents = step_ref.random_parents(np.random.default_rng(at), 2, T, wide=50)
    nodes = np.full(2, T)
    for b, L in enumerate(case.lens):
        enlarge(cache, b, L - T + at, by)
    check(cache, run(kvq, cache, parents), parents, nodes)


@pytest.mark.parametrize("name,T", [("int8 row d128", 6), ("int8 row d128", 33), ("int8 row d256 g6", 12), ("int4 row", 9),
                                    ("int4 group", 8)])
def test_a_large_row_behind_the_window(kvq, name, T):
    """A chain under a window: a large prefix row is seen by the first nodes only."""
    base = CASES[name]
    case = dataclasses.replace(base, c=T, lens=(300 + T, 90 + T), window=20, seed=T)
    cache = ref.Cache(case)
    parents = np.tile(np.arange(T, dtype=np.int32) - 1, (2, 1))
    nodes = np.full(2, T)
    for b, L in enumerate(case.lens):
        enlarge(cache, b, L - T - 17, 2.0 ** 30)  # nodes 0 .. 2 see it
    check(cache, run(kvq, cache, parents), parents, nodes)


@pytest.mark.parametrize("name,T,hq", [("int4 group", 4, 8), ("int4 group", 5, 2), ("int4 group", 20, 6),
                                       ("fp8 group v", 8, 2), ("fp8 group v", 9, 6), ("int8 group k, row v", 7, 6),
                                       ("latent d256", 5, 3), ("latent d576", 6, 8), ("latent d576", 4, 1)])
@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_a_node_of_group_scales_that_is_not_finite_reaches_its_descendants_only(kvq, name, T, hq, bad):
    """(An odd number of heads a group: two nodes share a lane's pair of rows.)"""
    cache, parents, nodes = make(name, T, ragged=False, hq=hq)
    parents[:, -1] = -1
    g = gpu_cache(kvq, cache)
    for b, L in enumerate(cache.case.lens):
        page, row = int(cache.table[b, (L - 1) // g.block_size]), (L - 1) % g.block_size
        if cache.case.km in (ref.ROW, ref.GROUP):
            g.k_scale[page, :, row] = bad
        if cache.case.vm in (ref.ROW, ref.GROUP) and not cache.case.latent:
            g.v_scale[page, :, row] = bad
    check(cache, run(kvq, cache, parents, gcache=g), parents, nodes, slice(0, T - 1))
