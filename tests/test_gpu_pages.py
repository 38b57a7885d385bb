"""The bookkeeping of pages (kvq_pages_step) against a plain stack of pages, and
a serving loop of all the step's calls.  Whole numbers: everything is equal."""
import numpy as np
import pytest
import torch

import step_ref
from guard import guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def dev(a, dt=np.int32):
    return guarded(torch.from_numpy(np.ascontiguousarray(np.asarray(a, dt))).cuda())


def run(kvq, ref, held, start, new, table, free, count, parents=None, in_place=False, nodes=0):
    """The call's outputs and flags."""
    B = len(held)
    p = kvq.make_pages_params(B, ref.width, num_blocks=ref.nb, block_size=ref.bs, max_tokens=ref.room,
                              tree_nodes=0 if parents is None else parents.shape[1])
    t = dict(held=dev(held), start=None if start is None else dev(start), new=dev(new), table=dev(table), free=dev(free),
             count=dev([count]), cu=dev(np.full(B + 1, 77)), slots=dev(np.full(ref.room, 77), np.int64),
             pos=dev(np.full(ref.room, 77), np.int64))
    lens = t["held"] if in_place else dev(np.full(B, 77))
    left = t["count"] if in_place else dev([77])
    kvq.kvq_pages_step(p, t["held"], t["start"], t["new"], None if parents is None else dev(parents), t["table"],
                       t["free"], t["count"], lens, left, t["cu"], t["slots"], t["pos"])
    flags = kvq.kvq_get_device_error()
    return [x.cpu().numpy() for x in (t["table"], t["free"], left, lens, t["cu"], t["slots"], t["pos"])] + [flags]


def check(got, want):
    names = ("block_table", "free_blocks", "free_left", "seq_lens", "cu_seqlens", "slot_mapping", "positions")
    for n, g, w in zip(names, got, want):
        assert np.array_equal(g, np.asarray(w).reshape(g.shape)), n
    assert got[7] == want[7]


def pool(r, held, bs, width, spare):
    """A table that holds the pages of `held` rows, and a free list of the rest."""
    need = [-(-int(h) // bs) for h in held]
    nb = max(1, sum(need) + spare)
    perm = r.permutation(nb).astype(np.int32)
    table, at = np.full((len(held), width), -9, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    free = np.full(nb, -7, np.int32)
    free[:spare] = perm[sum(need):][:spare]
    return nb, table, free


def scene(seed, B, bs, room=None, spare=None, tree=0, top=400):
    r = np.random.default_rng(seed)
    held = r.integers(0, top, B)
    held[r.random(B) < 0.2] = 0
    start = np.array([r.integers(0, h + 1) if r.random() < 0.5 else h for h in held])
    new = r.integers(0, top // 2, B)
    new[r.random(B) < 0.3] = 1
    done = r.random(B) < 0.15
    start[done], new[done] = 0, 0
    width = -(-(int((start + new).max(initial=1)) + top) // bs)
    up = lambda n: -(-n // bs)  # noqa: E731
    spare = int(np.maximum(0, up(start + new) - up(held)).sum()) if spare is None else spare
    nb, table, free = pool(r, held, bs, width, spare)
    ref = step_ref.Pages(bs, width, nb, int(new.sum()) + 5 if room is None else room)
    parents = step_ref.random_parents(r, B, tree) if tree else None
    return ref, held, start, new, table, free, spare, parents


@pytest.mark.parametrize("B", [1, 2, 31, 64, 257, 1024])
@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_of_many_kinds(kvq, B, bs, in_place):
    ref, *x, parents = scene(B + bs, B, bs)
    check(run(kvq, ref, *x, in_place=in_place), ref.step(*x))


@pytest.mark.parametrize("B,tree", [(1, 1), (5, 9), (64, 64), (300, 13), (20, 256)])
def test_positions_of_trees(kvq, B, tree):
    """Nodes get the position of their depth; tokens behind the tree their row."""
    ref, *x, parents = scene(7 * B, B, 16, tree=tree)
    check(run(kvq, ref, *x, parents=parents), ref.step(*x, parents=parents))


@pytest.mark.parametrize("seed", range(12))
def test_short_pools_and_short_slot_maps(kvq, seed):
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 200))
    ref, *x, _ = scene(seed, B, 16)
    spare = int(x[-1])
    small = scene(seed, B, 16, spare=int(r.integers(0, spare + 1)), room=int(r.integers(0, ref.room)) if seed % 2 else None)
    ref, *x, _ = small
    check(run(kvq, ref, *x, in_place=seed % 3 == 0), ref.step(*x))


@pytest.mark.parametrize("tokens", [0, 1, 1023, 1024, 1025, 4096, 4097, 100000])
def test_one_prompt_of_any_length(kvq, tokens):
    ref = step_ref.Pages(16, 8000, 7000, tokens + (3 if tokens % 2 else 0))
    table, free = np.full((1, 8000), -9, np.int32), np.arange(7000)[::-1].astype(np.int32)
    x = [0], [0], [tokens], table, free, 7000
    check(run(kvq, ref, *x), ref.step(*x))


def test_start_lens_may_be_left_out(kvq):
    ref, held, start, new, *rest, _ = scene(3, 40, 16, spare=2000)
    got = run(kvq, ref, held, None, new, *rest)
    check(got, ref.step(held, held, new, *rest))


def test_impossible_lengths_are_refused_and_flagged(kvq):
    """Negative lengths, starts behind the held rows, rows past the table, sums
    past 32 bits: those sequences stay as they were, the others get theirs."""
    top = 2 ** 31 - 1
    held = np.array([30, -1, 30, 30, 0, 16 * 40, 16 * 40 + 1, 5, 30, top, 20])
    start = np.array([30, 0, 31, -2, 0, 0, 0, 5, 30, 0, 3])
    new = np.array([1, 1, 1, 1, 16 * 40 + 1, 0, 1, top, -1, top, 50])
    r = np.random.default_rng(0)
    bs, width = 16, 40
    nb, table, free = pool(r, np.where((held < 0) | (held > bs * width), 0, held), bs, width, 50)
    ref = step_ref.Pages(bs, width, nb, 2 ** 20)
    x = held, start, np.array(new), table, free, 50
    got, want = run(kvq, ref, *x), ref.step(*x)
    check(got, want)
    assert want[7] == ref.SEQ_LEN
    # the token counts past the map's room refuse all that come behind them
    assert list(want[3][[7, 10]]) == [5, 20] and want[3][0] == 31


def test_bad_page_ids_are_passed_on_and_flagged(kvq):
    r = np.random.default_rng(1)
    held, start, new = np.array([64, 0, 20]), np.array([0, 0, 20]), np.array([0, 70, 3])
    nb, table, free = pool(r, held, 16, 8, 3)
    ref = step_ref.Pages(16, 8, nb, 100)
    for bad in (-1, nb, 2 ** 31 - 1, -(2 ** 31)):
        t, f = table.copy(), free.copy()
        t[0, 3], f[1] = bad, bad
        x = held, start, new, t, f, 3
        want = ref.step(*x)
        assert want[7] == ref.BLOCK_ID
        check(run(kvq, ref, *x), want)


def test_counts_outside_the_pool_are_flagged(kvq):
    held, new = np.array([0]), np.array([20])
    table, free = np.full((1, 4), -9, np.int32), np.arange(6, dtype=np.int32)
    ref = step_ref.Pages(16, 4, 6, 32)
    for count, cut in ((-3, 0), (7, 6), (2 ** 31 - 1, 6)):
        got, want = run(kvq, ref, held, held, new, table, free, count), ref.step(held, held, new, table, free, cut)
        assert got[7] == want[7] | ref.BLOCK_ID
        check(got[:7] + [want[7]], want)
    # more pages given back than the pool has: the surplus is not taken
    held = np.array([64, 64])
    t = np.tile(np.arange(4, dtype=np.int32), (2, 1))
    got = run(kvq, step_ref.Pages(16, 4, 6, 8), held, [0, 0], [0, 0], t, np.full(6, -7, np.int32), 1)
    assert got[7] == ref.BLOCK_ID and got[2] == 6 and list(got[1]) == [-7, 0, 1, 2, 3, 0]


def test_a_pool_lives_through_many_steps(kvq):
    """A hundred steps in place under one captured graph: no page is lost or
    held twice, whatever comes and goes."""
    r = np.random.default_rng(11)
    B, bs, width, nb, room = 24, 16, 20, 200, 1500
    ref = step_ref.Pages(bs, width, nb, room)
    p = kvq.make_pages_params(B, width, num_blocks=nb, block_size=bs, max_tokens=room)
    t_len, t_start, t_new = (dev(np.zeros(B)) for _ in range(3))
    t_table, t_free, t_count = dev(np.full((B, width), -9)), dev(r.permutation(nb)), dev([nb])
    t_cu, t_slots, t_pos = dev(np.zeros(B + 1)), dev(np.zeros(room), np.int64), dev(np.zeros(room), np.int64)
    table, free, count, lens = t_table.cpu().numpy(), t_free.cpu().numpy(), nb, np.zeros(B, np.int32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_pages_step(p, t_len, t_start, t_new, None, t_table, t_free, t_count, t_len, t_count, t_cu, t_slots, t_pos)
    refused = 0
    for _ in range(100):
        start = np.array([0 if r.random() < 0.1 else r.integers(max(0, n - 20), n + 1) for n in lens], np.int32)
        new = np.where(start > 0, r.integers(0, 30, B), r.integers(0, 250, B) * (r.random(B) < 0.5)).astype(np.int32)
        t_start.copy_(torch.from_numpy(start)); t_new.copy_(torch.from_numpy(new))
        graph.replay()
        table, free, count, lens, cu, slots, pos, flags = ref.step(lens, start, new, table, free, count)
        check([x.cpu().numpy() for x in (t_table, t_free, t_count, t_len, t_cu, t_slots, t_pos)]
              + [kvq.kvq_get_device_error()], [table, free, count, lens, cu, slots, pos, flags])
        held = [int(table[b, i]) for b in range(B) for i in range(-(-int(lens[b]) // bs))]
        assert sorted(held + [int(x) for x in free[:count]]) == list(range(nb))
        refused += flags != 0
    assert 0 < refused < 100


def test_a_serving_loop(kvq):
    """Prompts, then drafted trees: pages, append, prompt attention, tree
    attention and acceptance one after another without a host round trip.  The
    cache ends as if only the accepted tokens had ever been appended."""
    r = np.random.default_rng(8)
    B, T, hq, hkv, d, bs, width, nb = 5, 7, 8, 2, 128, 16, 12, 80
    room = 512
    cache = kvq.QuantizedPagedCache(kvq.INT8, kvq.PER_ROW, kvq.PER_ROW, nb, bs, hkv, d)
    pages = kvq.make_pages_params(B, width, num_blocks=nb, block_size=bs, max_tokens=room, tree_nodes=T)
    lens, start, zeros = dev(np.zeros(B)), dev(np.zeros(B)), dev(np.zeros(B))
    table, free, count = dev(np.full((B, width), -9)), dev(r.permutation(nb)), dev([nb])
    cu, slots, pos = dev(np.zeros(B + 1)), dev(np.zeros(room), np.int64), dev(np.zeros(room), np.int64)
    bf = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
    torch.manual_seed(3)

    prompts = np.array([33, 1, 64, 100, 17])
    kvq.kvq_pages_step(pages, lens, None, dev(prompts), None, table, free, count, lens, count, cu, slots, pos)
    k, v, q = bf(room, hkv, d), bf(room, hkv, d), bf(room, hq, d)
    kvq.kvq_append(cache, k, v, slots)
    pp = kvq.make_prompt_params(B, room, hq, hkv, d)
    pws = torch.empty(kvq.kvq_attend_prompt_workspace_size(pp) // 4, dtype=torch.int32, device="cuda")
    pout, plse = torch.zeros((room, hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((room, hq), device="cuda")
    kvq.kvq_attend_prompt(pp, q, k, v, cu, None, pout, plse, pws)
    # the same last tokens over the quantized cache: the int8 rounding apart
    # (half a step of absmax / 127 a value: about 1% of a normal row's size)
    ends = np.cumsum(prompts) - 1
    dp = kvq.make_params(B, hq, 1, width)
    bufs = kvq.alloc_decode_buffers(cache, dp)
    dout, dlse = kvq.decode_step(cache, dp, q[ends].reshape(B, 1, hq, d).contiguous(), table, lens, bufs)
    a, b = pout[ends].float(), dout[:, 0].float()
    assert (a - b).norm() / a.norm() < 0.02 and (plse[ends] - dlse[:, 0]).abs().max() < 0.05
    said = [list(range(int(s), int(e) + 1)) for s, e in zip(np.cumsum(prompts) - prompts, ends)]
    rows = [(k[i].clone(), v[i].clone()) for i in said]  # the rows each sequence should hold

    tp = kvq.make_params(B, hq, T, width)
    tws = torch.empty(kvq.kvq_attend_tree_workspace_size(cache, tp) // 4, dtype=torch.int32, device="cuda")
    out, lse = torch.empty((B, T, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, T, hq), device="cuda")
    path, acc, nxt = dev(np.zeros((B, T))), dev(np.zeros(B)), dev(np.zeros(B), np.int64)
    start.copy_(lens)
    grown = []
    for step in range(6):
        parents = step_ref.random_parents(r, B, T, wide=3)
        nodes = r.integers(1, T + 1, B).astype(np.int32)
        drafts = r.integers(0, 3, (B, T)).astype(np.int64)
        chosen = r.integers(0, 3, (B, T)).astype(np.int64)
        t_par, t_n = dev(parents), dev(nodes)
        k, v, q = bf(room, hkv, d), bf(room, hkv, d), bf(B, T, hq, d)
        kvq.kvq_pages_step(pages, lens, start, t_n, t_par, table, free, count, lens, count, cu, slots, pos)
        kvq.kvq_append(cache, k, v, slots)
        tree = kvq.DraftTree(t_par, t_n)
        kvq.kvq_attend_tree(cache, tp, tree, q, table, lens, None, out, lse, tws)
        kvq.kvq_tree_accept(cache, tp, tree, dev(drafts, np.int64), dev(chosen, np.int64), table, lens, path, acc, start, nxt)
        at = np.concatenate([[0], np.cumsum(nodes)])
        paths, after = step_ref.accept(parents, nodes, drafts, chosen)
        for b, p in enumerate(paths):
            i = [int(at[b]) + n for n in p]
            rows[b] = (torch.cat([rows[b][0], k[i]]), torch.cat([rows[b][1], v[i]]))
        grown.append(max(len(p) for p in paths))
        assert nxt.tolist() == after and start.tolist() == [x[0].shape[0] for x in rows]
        assert torch.isfinite(out.float()).all()
    assert max(grown) > 2 and kvq.kvq_get_device_error() == 0
    plain = kvq.QuantizedPagedCache(kvq.INT8, kvq.PER_ROW, kvq.PER_ROW, nb, bs, hkv, d)
    for b, (kk, vv) in enumerate(rows):
        i = torch.arange(kk.shape[0], device="cuda")
        slot = table[b, i // bs].long() * bs + i % bs
        kvq.kvq_append(plain, kk.contiguous(), vv.contiguous(), slot)
        blk, row = table[b, i // bs].long(), i % bs
        for x in ("k_codes", "v_codes", "k_scale", "v_scale"):
            assert torch.equal(getattr(cache, x)[blk, :, row], getattr(plain, x)[blk, :, row]), x
