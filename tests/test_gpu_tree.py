"""Attention of draft trees (kvq_attend_tree) against its 64-bit form, and the
accepted paths with the move of their rows (kvq_tree_accept) against a plain
walk.

Tolerances of the attention are those of test_gpu_masked (the kernels are the
same): bf16 rounding of the result 2^-8 of it, f16 weights and scaled values
(step_ref.attend_tree adds these up), a logit off by at most 2^-11 of
sum |q k| when a per-channel K scale is folded into an f16 query, else 2^-15,
which moves the result by at most twice that times sum p |v|."""
import dataclasses

import numpy as np
import pytest
import torch

import score_ref as ref
import step_ref
from guard import guarded
from test_gpu_masked import CASES, dev, gpu_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def run(kvq, c: ref.Cache, parents, nodes=None, sink=None, lse=True, flags=0, err=0, gcache=None, lens=None):
    case = c.case
    g = gcache or gpu_cache(kvq, c)
    B = len(case.lens)
    p = kvq.make_params(B, case.hq, case.c, c.width, softcap=case.softcap, window=case.window,
                        sm_scale=case.sm_scale, flags=flags)
    ws = guarded(torch.full((kvq.kvq_attend_tree_workspace_size(g, p) // 4,), -1, dtype=torch.int32, device="cuda"), "ws")
    out = guarded(torch.full((B, case.c, case.hq, g.out_dim), 7.0, dtype=torch.bfloat16, device="cuda"), "out")
    l = guarded(torch.full((B, case.c, case.hq), 7.0, device="cuda"), "lse") if lse else None
    tree = kvq.DraftTree(dev(parents), None if nodes is None else dev(np.asarray(nodes, np.int32)))
    kvq.kvq_attend_tree(g, p, tree, dev(c.q).to(torch.bfloat16), dev(c.table),
                        dev(np.array(case.lens if lens is None else lens, np.int32)),
                        None if sink is None else dev(np.asarray(sink, np.float32)), out, l, ws)
    assert kvq.kvq_get_device_error() == err
    return out.float().cpu().numpy().astype(np.float64), None if l is None else l.cpu().numpy().astype(np.float64)


def check(c: ref.Cache, got, parents, nodes, sink=None):
    out, lse = got
    r_out, r_lse, absv, f16, size = step_ref.attend_tree(c, parents, nodes, sink)
    ds = (2.0 ** -11 * size if c.case.km == step_ref.CHANNEL else np.zeros_like(size)) + 2.0 ** -15
    empty = r_lse == -np.inf
    if lse is not None:
        assert (lse[empty] == -np.inf).all() and np.isfinite(lse[~empty]).all()
        e = np.abs(lse[~empty] - r_lse[~empty]) - (ds[~empty] + 2.0 ** -20 * (1 + np.abs(r_lse[~empty])))
        assert e.size == 0 or e.max() <= 0, f"lse off by {e.max():.2e} more than its bound"
    assert (out[empty] == 0).all() and np.isfinite(out).all()
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    worst = (np.abs(out - r_out) / tol).max()
    assert worst <= 1.0, f"output {worst:.2f} times its bound"


def make(name, T, seed=0, ragged=True, **kw):
    base = CASES[name]
    r = np.random.default_rng(seed + 3 * T)
    lens = tuple(max(L, T + 3) for L in base.lens)
    case = dataclasses.replace(base, c=T, seed=seed + T, lens=lens, **kw)
    parents = step_ref.random_parents(r, len(lens), T)
    nodes = r.integers(1, T + 1, len(lens)) if ragged else np.full(len(lens), T)
    return ref.Cache(case), parents, nodes


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("T", [1, 5, 13, 33, 70])
def test_random_trees(kvq, name, T):
    cache, parents, nodes = make(name, T)
    check(cache, run(kvq, cache, parents, nodes), parents, nodes)


@pytest.mark.parametrize("name", ["int8 row d128", "fp8 tensor cap", "int4 channel d256", "int8 channel d64", "latent d576"])
@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("window", [1, 4, 30, 64])
def test_windows_and_sinks(kvq, name, T, window):
    """Windows smaller than a chain cut its far ancestors; larger ones the prefix."""
    cache, parents, nodes = make(name, T, seed=window, window=window)
    sink = np.linspace(-1, 2, cache.case.hq)
    check(cache, run(kvq, cache, parents, nodes, sink), parents, nodes, sink)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 row d256 g6", "int4 channel d256", "int8 channel d64"])
@pytest.mark.parametrize("T", [7, 64])
def test_without_lse_and_without_tensor_memory(kvq, name, T):
    cache, parents, nodes = make(name, T, ragged=False)
    check(cache, run(kvq, cache, parents, lse=False), parents, nodes)
    check(cache, run(kvq, cache, parents, flags=kvq.DECODE_NO_TCGEN05), parents, nodes)


@pytest.mark.parametrize("name,T", [("int8 row d128", 5), ("int8 row d128", 40), ("fp8 row", 3), ("int4 row", 17)])
def test_trees_over_no_prefix_and_empty_sequences(kvq, name, T):
    """All rows are nodes; one sequence has no nodes over a prefix, one no rows."""
    case = dataclasses.replace(CASES[name], c=T, lens=(T, T - 1, 50, 0, T), seed=T)
    cache = ref.Cache(case)
    parents = step_ref.random_parents(np.random.default_rng(T), 5, T)
    nodes = np.array([T, T - 1, 0, 0, 1])
    check(cache, run(kvq, cache, parents, nodes), parents, nodes)


@pytest.mark.parametrize("name", ["int8 row d128", "fp8 tensor cap", "int8 row d256 g6", "int4 channel d256"])
@pytest.mark.parametrize("T", [3, 13])
def test_trees_over_long_prefixes(kvq, name, T):
    """Many tiles of many CTAs, one sequence beside it that is shorter than a tile."""
    base = CASES[name]
    case = dataclasses.replace(base, c=T, seed=T, lens=(8009, 63 + T))
    cache = ref.Cache(case)
    parents = step_ref.random_parents(np.random.default_rng(T), 2, T)
    nodes = np.array([T, (T + 1) // 2])
    check(cache, run(kvq, cache, parents, nodes), parents, nodes)


@pytest.mark.parametrize("name,T", [("int8 row d128", 2), ("int8 row d128", 5), ("int8 row d128", 40),
                                    ("int8 row d256 g6", 16), ("fp8 row", 20), ("int4 row", 3), ("int4 row", 33)])
@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_a_node_that_is_not_finite_reaches_its_descendants_only(kvq, name, T, bad):
    cache, parents, nodes = make(name, T, ragged=False)
    parents[:, -1] = -1  # the last node: a root without children, seen by itself alone
    g = gpu_cache(kvq, cache)
    for b, L in enumerate(cache.case.lens):
        page, row = cache.table[b, (L - 1) // g.block_size], (L - 1) % g.block_size
        g.k_scale[int(page), :, row] = bad
        g.v_scale[int(page), :, row] = bad
    out, lse = run(kvq, cache, parents, gcache=g)
    r_out, r_lse, absv, f16, size = step_ref.attend_tree(cache, parents, nodes, None)
    seen, ds = slice(0, T - 1), 2.0 ** -15
    assert np.isfinite(out[:, seen]).all() and np.isfinite(lse[:, seen]).all()
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds * absv + 1e-30
    assert (np.abs(out - r_out) / tol)[:, seen].max() <= 1.0
    assert (np.abs(lse - r_lse) <= ds + 2.0 ** -20 * (1 + np.abs(r_lse)))[:, seen].all()


@pytest.mark.parametrize("name,T", [("int8 row d128", 256), ("fp8 tensor cap", 200)])
def test_the_largest_trees(kvq, name, T):
    """A tree of 256 nodes, among them a chain of all of them."""
    cache, parents, nodes = make(name, T, ragged=False)
    parents[0] = np.arange(T) - 1
    check(cache, run(kvq, cache, parents), parents, nodes)


@pytest.mark.parametrize("name", ["int8 row d128", "int4 channel d256", "fp8 row"])
@pytest.mark.parametrize("T", [4, 30])
def test_a_chain_is_causal_attention(kvq, name, T):
    """One chain of nodes sees what T causal tokens see (window included)."""
    from test_gpu_masked import check as check_masked
    cache, _, _ = make(name, T, window=45)
    parents = np.tile(np.arange(T, dtype=np.int32) - 1, (len(cache.case.lens), 1))
    got = run(kvq, cache, parents)
    check(cache, got, parents, np.full(len(cache.case.lens), T))
    check_masked(cache, got)


def test_node_counts_outside_their_range_are_flagged(kvq):
    cache, parents, _ = make("int8 row d128", 9)
    B = len(cache.case.lens)
    got = run(kvq, cache, parents, [-3, 12, 9], err=kvq.DEVERR_SEQ_LEN)
    check(cache, got, parents, np.array([0, 9, 9][:B]))


def test_seams_of_tiles_and_pages(kvq):
    """The prefix ends at, before and behind tiles of 64 keys; trees cross them."""
    for P in (0, 1, 15, 16, 31, 63, 64, 65, 127, 128, 129):
        case = dataclasses.replace(CASES["int8 row d128"], c=37, lens=(P + 37, P + 20), seed=P)
        cache = ref.Cache(case)
        parents = step_ref.random_parents(np.random.default_rng(P), 2, 37)
        nodes = np.array([37, 20])
        check(cache, run(kvq, cache, parents, nodes), parents, nodes)
        case = dataclasses.replace(case, c=2, lens=(P + 2, P + 1), seed=P)
        cache = ref.Cache(case)
        check(cache, run(kvq, cache, parents[:, :2].copy(), [2, 1]), parents[:, :2], [2, 1])


def test_repeated_calls_streams_and_graphs_give_the_same_bits(kvq):
    cache, parents, nodes = make("int8 row d256 g6", 19)
    g = gpu_cache(kvq, cache)
    first = run(kvq, cache, parents, nodes, gcache=g)
    with torch.cuda.stream(torch.cuda.Stream()):
        again = run(kvq, cache, parents, nodes, gcache=g)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    case = cache.case
    B = len(case.lens)
    p = kvq.make_params(B, case.hq, case.c, cache.width)
    ws = torch.empty(kvq.kvq_attend_tree_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    q, table = dev(cache.q).to(torch.bfloat16), dev(cache.table)
    par, n, lens = dev(np.zeros_like(parents)), dev(np.zeros(B, np.int32)), dev(np.zeros(B, np.int32))
    out = torch.empty((B, case.c, case.hq, case.d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, case.c, case.hq), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_attend_tree(g, p, kvq.DraftTree(par, n), q, table, lens, None, out, lse, ws)
    par.copy_(dev(parents)); n.copy_(dev(nodes.astype(np.int32))); lens.copy_(dev(np.array(case.lens, np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.float().cpu().numpy(), first[0]) and np.array_equal(lse.cpu().numpy(), first[1])


# ------------------------------------------------------------------ accept

def accept(kvq, c: ref.Cache, g, parents, nodes, drafts, chosen, mass=None, err=0, lens=None, table=None):
    case = c.case
    B, T = parents.shape
    p = kvq.make_params(B, case.hq, T, c.width)
    full = lambda shape, dt: guarded(torch.full(shape, 77, dtype=dt, device="cuda"))  # noqa: E731
    path, acc, new, nxt = (full((B, T), torch.int32), full((B,), torch.int32), full((B,), torch.int32),
                           full((B,), torch.int64))
    tree = kvq.DraftTree(dev(parents), None if nodes is None else dev(np.asarray(nodes, np.int32)))
    kvq.kvq_tree_accept(g, p, tree, dev(drafts), dev(chosen), dev(c.table if table is None else table),
                        dev(np.array(case.lens if lens is None else lens, np.int32)), path, acc, new, nxt, mass)
    assert kvq.kvq_get_device_error() == err
    return [t.cpu().numpy() for t in (path, acc, new, nxt)]


def likely(r, parents, vocab=7, follow=0.85):
    """Drafted tokens and choices that often agree with one of the children."""
    B, T = parents.shape
    drafts = r.integers(0, vocab, (B, T)).astype(np.int64)
    drafts += (1 << 40) * r.integers(0, 2, (B, T))  # tokens that differ above 32 bits only
    chosen = r.integers(0, vocab, (B, T)).astype(np.int64)
    for b in range(B):
        for i in range(T):
            kids = [j for j in range(i + 1, T) if parents[b, j] == i]
            if kids and (i == 0 or r.random() < follow):
                chosen[b, i] = drafts[b, r.choice(kids)]
    return drafts, chosen


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("T", [1, 6, 40, 130])
def test_accepted_rows_move_together(kvq, name, T):
    cache, parents, nodes = make(name, T, seed=5)
    case, r = cache.case, np.random.default_rng(T)
    nodes = nodes.copy()
    if len(nodes) > 1:
        nodes[-1] = 0
    drafts, chosen = likely(r, parents, follow=0.97 if T > 40 else 0.85)
    g = gpu_cache(kvq, cache)
    mass = guarded(torch.rand((cache.nb, case.hkv, case.bs), device="cuda"), "mass")
    arrays = [g.k_codes, g.v_codes, mass]
    arrays += [g.k_scale] if case.km in (ref.ROW, ref.GROUP) else []
    arrays += [g.v_scale] if case.vm in (ref.ROW, ref.GROUP) and not case.latent else []
    before = [a.view(torch.uint8).cpu().numpy().copy() for a in arrays]
    path, acc, new, nxt = accept(kvq, cache, g, parents, nodes, drafts, chosen, mass)
    want, after = step_ref.accept(parents, nodes, drafts, chosen)
    for b, p in enumerate(want):
        P = case.lens[b] - int(nodes[b])
        assert list(path[b]) == p + [-1] * (T - len(p)) and acc[b] == len(p) and new[b] == P + len(p)
        assert nxt[b] == after[b]
    moved = [w.copy() for w in before]
    for b, p in enumerate(want):
        P = case.lens[b] - int(nodes[b])
        for i, n in enumerate(p):
            (sb, sr), (db, dr) = ((cache.table[b, x // case.bs], x % case.bs) for x in (P + n, P + i))
            for m, w in zip(moved, before):
                per = m.shape[-1] // case.bs if m.ndim == 3 else None
                if per:  # [blocks, heads, rows * bytes]
                    m[db, :, dr * per:(dr + 1) * per] = w[sb, :, sr * per:(sr + 1) * per]
                else:
                    m[db, :, dr] = w[sb, :, sr]
    for a, m in zip(arrays, moved):
        assert np.array_equal(a.view(torch.uint8).cpu().numpy(), m)


def test_the_lowest_of_equal_children_is_accepted(kvq):
    case = dataclasses.replace(CASES["int8 row d128"], c=5, lens=(20,))
    cache = ref.Cache(case)
    parents = np.array([[-1, 0, 0, 1, 2]], np.int32)
    drafts, chosen = np.array([[9, 4, 4, 8, 8]]), np.array([[4, 8, 8, 1, 2]])
    path, acc, new, nxt = accept(kvq, cache, gpu_cache(kvq, cache), parents, None, drafts, chosen)
    assert list(path[0]) == [0, 1, 3, -1, -1] and acc[0] == 3 and new[0] == 18 and nxt[0] == 1


def test_unreadable_pages_of_nodes_are_flagged_and_not_moved(kvq):
    case = dataclasses.replace(CASES["int8 row d128"], c=20, lens=(40, 40), bs=16)
    cache = ref.Cache(case)
    parents = np.full((2, 20), -1, np.int32)
    parents[:, 18], parents[:, 19] = 0, 18
    drafts, chosen = np.zeros((2, 20), np.int64), np.zeros((2, 20), np.int64)
    g = gpu_cache(kvq, cache)
    table = cache.table.copy()
    table[0, 2], table[1, 1] = cache.nb, -5  # rows 32..47 of the first, 16..31 of the second
    k = g.k_codes.clone()
    path, acc, new, _ = accept(kvq, cache, g, parents, None, drafts, chosen, err=kvq.DEVERR_BLOCK_ID, table=table)
    assert list(acc) == [3, 3] and list(new) == [23, 23] and list(path[0, :3]) == [0, 18, 19]
    assert torch.equal(g.k_codes, k)  # sources 38, 39 of the first and rows 21, 22 of the second are unreadable


def test_lengths_outside_their_range_are_flagged(kvq):
    cache, parents, _ = make("int8 row d128", 6)
    B = len(cache.case.lens)
    drafts = np.zeros((B, 6), np.int64)
    g = gpu_cache(kvq, cache)
    _, acc, new, nxt = accept(kvq, cache, g, parents, None, drafts, drafts + 1, err=kvq.DEVERR_SEQ_LEN,
                              lens=[-4, 2 ** 31 - 1, 3])
    assert acc[0] == 0 and new[0] == 0 and nxt[0] == -1
    assert acc[1] == 1 and new[1] == cache.width * cache.case.bs - 6 + 1
    assert acc[2] == 1 and new[2] == 1  # three rows: three nodes
