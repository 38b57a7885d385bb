"""Evictions as a serving loop runs them, and selections at the edges of what
the arguments allow, against the plain forms of score_ref."""
import numpy as np
import pytest
import torch

import score_ref as ref
from guard import guarded
from test_gpu_evict import masses, pages, select_call
from test_gpu_masked import dev

pytestmark = pytest.mark.gpu

INT8, ROW = ref.INT8, ref.ROW


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


@pytest.mark.parametrize("add", ["in place", "out of place", "none"])
def test_lengths_stay_on_the_device(kvq, add):
    """seq_lens = evict_step(...) step after step with the same buffers: the
    returned lengths are the next step's argument, as they are, advanced in
    place, or through a new tensor."""
    hkv, d, bs, budget, width, nb = 2, 64, 16, 40, 4, 10
    r = np.random.default_rng(3)
    table = r.permutation(nb)[:2 * width].reshape(2, width).astype(np.int32)
    g = kvq.QuantizedPagedCache(INT8, ROW, ROW, nb, bs, hkv, d)
    for t in (g.k_codes, g.v_codes):
        t.copy_(dev(r.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
    ep = kvq.make_evict_params(2, width, budget, num_blocks=nb, block_size=bs, num_kv_heads=hkv, sinks=2, recent=4)
    bufs = kvq.alloc_evict_buffers(g, ep)
    tbl, lens = dev(table), np.array([64, 50], np.int32)
    seq_lens = dev(lens)
    for step in range(5):
        mass = dev(r.exponential(0.1, (nb, hkv, bs)).astype(np.float32))
        want, kept = ref.select(mass.cpu().numpy(), table, [int(x) for x in lens], bs, budget, 2, 4)
        arrays = [t.cpu().numpy() for t in (g.k_codes, g.v_codes, g.k_scale, g.v_scale, mass)]
        moved = ref.compact(arrays, table, table, want, kept, bs)
        given = seq_lens.clone()
        before = seq_lens
        seq_lens = kvq.evict_step(g, ep, tbl, seq_lens, mass, bufs)
        assert torch.equal(before, given), "the lengths that were passed changed"
        assert np.array_equal(seq_lens.cpu().numpy(), kept)
        assert np.array_equal(bufs.keep.cpu().numpy(), want)
        for t, w in zip((g.k_codes, g.v_codes, g.k_scale, g.v_scale, mass), moved):
            assert np.array_equal(t.cpu().numpy(), w)
        lens = kept
        if add != "none":
            n = 9 + step
            seq_lens = seq_lens.add_(n) if add == "in place" else seq_lens + n
            lens = kept + np.int32(n)
    assert kvq.kvq_get_device_error() == 0


def test_lengths_beside_one_another(kvq):
    """seq_lens, kept_lens and keep in one allocation, end to end: nothing overlaps."""
    bs, hkv, budget, lens = 16, 3, 50, (200, 17, 90)
    table, nb = pages(lens, bs, 1)
    mass = masses("weights", hkv, bs)(nb)
    n = hkv * budget
    one = guarded(torch.zeros(3 + 3 + 3 * n, dtype=torch.int32, device="cuda"), "lengths and rows")
    one[:3].copy_(dev(np.array(lens, np.int32)))
    p = kvq.make_evict_params(3, table.shape[1], budget, num_blocks=nb, block_size=bs, num_kv_heads=hkv)
    keep = one[6:].view(3, hkv, budget)
    kvq.kvq_evict_select(p, dev(mass), dev(table), one[:3], keep, one[3:6])
    assert kvq.kvq_get_device_error() == 0
    want = ref.select(mass, table, lens, bs, budget, 0, 0)
    assert np.array_equal(keep.cpu().numpy(), want[0]) and np.array_equal(one[3:6].cpu().numpy(), want[1])


def test_rows_in_the_workspace_are_refused(kvq):
    """The rows' places may not lie in the part of the workspace that a call uses;
    behind it, in the same allocation, they may."""
    bs, hkv, d, budget, lens = 16, 2, 64, 24, (60, 33)
    g = kvq.QuantizedPagedCache(INT8, ROW, ROW, 10, bs, hkv, d)
    p = kvq.make_evict_params(2, 4, budget, num_blocks=10, block_size=bs, num_kv_heads=hkv)
    n = kvq.kvq_evict_compact_workspace_size(g, p) // 4
    arena = torch.zeros(n + 4 * 64, dtype=torch.int32, device="cuda")
    table = dev(np.arange(8, dtype=np.int32).reshape(2, 4))
    mass = torch.rand((10, hkv, bs), device="cuda")
    for at in (n, n - 1, 0):
        kept = arena[at:at + 2]
        keep = torch.zeros((2, hkv, budget), dtype=torch.int32, device="cuda")
        kvq.kvq_evict_select(p, mass, table, dev(np.array(lens, np.int32)), keep, kept)
        if at == n:
            kvq.kvq_evict_compact(g, p, table, None, keep, kept, mass, arena)
            assert kept.tolist() == [budget, budget]
        else:
            with pytest.raises(kvq.KvqError):
                kvq.kvq_evict_compact(g, p, table, None, keep, kept, mass, arena)
    assert kvq.kvq_get_device_error() == 0


def test_selection_while_the_weights_change(kvq):
    """Heads too long to be held on chip are read again in every pass.  Weights
    that another stream writes meanwhile make the rows in `keep` unspecified,
    but nothing outside their places is written: not the protected rows of the
    same head, and not what lies around keep."""
    bs, L, budget, sinks, recent = 1024, 600_000, 150_000, 7, 90
    table, nb = pages((L,), bs, 1)
    r = np.random.default_rng(0)
    kinds = [torch.from_numpy(r.exponential(1.0, (nb, 1, bs)).astype(np.float32)).cuda() for _ in range(3)]
    kinds.append(torch.zeros((nb, 1, bs), device="cuda"))
    kinds.append(torch.full((nb, 1, bs), 7.0, device="cuda"))
    mass = kinds[0].clone()
    p = kvq.make_evict_params(1, table.shape[1], budget, num_blocks=nb, block_size=bs, num_kv_heads=1, sinks=sinks,
                              recent=recent)
    keep = guarded(torch.full((1, 1, budget), -9, dtype=torch.int32, device="cuda"), "keep")
    kept = guarded(torch.zeros(1, dtype=torch.int32, device="cuda"), "kept")
    tbl, lens = dev(table), dev(np.array([L], np.int32))
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(other):
            for k in kinds * 4:
                mass.copy_(k)
        with torch.cuda.stream(mine):
            for _ in range(10):
                kvq.kvq_evict_select(p, mass, tbl, lens, keep, kept)
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_error() == 0
    ends = keep[0, 0].cpu().numpy()
    assert np.array_equal(ends[:sinks], np.arange(sinks))
    assert np.array_equal(ends[budget - recent:], np.arange(L - recent, L))
    mid = ends[sinks:budget - recent]
    assert ((mid == -9) | ((mid >= sinks) & (mid < L - recent))).all()
    # and left alone it is right again
    mass.copy_(kinds[0])
    kvq.kvq_evict_select(p, mass, tbl, lens, keep, kept)
    j = np.arange(sinks, L - recent)
    w = kinds[0].cpu().numpy()[table[0, j // bs], 0, j % bs]
    want = np.sort(j[np.lexsort((j, -w))[:budget - sinks - recent]])
    assert np.array_equal(keep[0, 0, sinks:budget - recent].cpu().numpy(), want)


FIRST_SELECTIONS = """
import threading
import numpy as np
import torch
from decode_attention_quantized_gb300 import kvq

kvq.load()
torch.cuda.init()
n, bs, L, budget = 8, 64, 20000, 777
nb = (L + bs - 1) // bs
mass = torch.rand((nb, 1, bs), device="cuda")
table = torch.randperm(nb, device="cuda", dtype=torch.int32).view(1, nb)
lens = torch.tensor([L], dtype=torch.int32, device="cuda")
keep = [torch.zeros((1, 1, budget), dtype=torch.int32, device="cuda") for _ in range(n)]
kept = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(n)]
p = kvq.make_evict_params(1, nb, budget, num_blocks=nb, block_size=bs, num_kv_heads=1)
torch.cuda.synchronize()
gate, failed = threading.Barrier(n), []

def call(i):
    try:
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        gate.wait()
        kvq.kvq_evict_select(p, mass, table, lens, keep[i], kept[i], stream=s)
        s.synchronize()
    except Exception as e:
        failed.append(e)

threads = [threading.Thread(target=call, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
w = mass.cpu().numpy()[table[0].cpu().numpy()][:, 0].reshape(-1)[:L]
want = np.sort(np.lexsort((np.arange(L), -w))[:budget])
for k in keep:
    assert np.array_equal(k[0, 0].cpu().numpy(), want)
assert kvq.kvq_get_device_error() == 0
print("first selections agree")
"""


def test_first_selections_of_several_threads(kvq):
    """Host threads whose selections are a process's first ones (in a process of
    their own) set the kernel's attributes side by side."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_SELECTIONS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first selections agree" in r.stdout, r.stderr


@pytest.mark.parametrize("batch", [129, 200])
def test_select_of_many_sequences(kvq, batch):
    """More than 128 sequences of unequal lengths in the one-pass selection
    (capacity of 40,960 rows, a head or more per SM): heads in batch order."""
    bs, hkv, budget, sinks, recent = 256, 2, 700, 3, 20
    r = np.random.default_rng(batch)
    lens = [int(x) for x in np.exp(r.uniform(np.log(2), np.log(9000), batch))]
    lens[5], lens[batch - 1], lens[77], lens[3] = 40960, 33000, 0, 700
    table, nb = pages(lens, bs, 2, width=160)
    mass = masses("weights", hkv, bs, 4)(nb)
    keep, kept = select_call(kvq, mass, table, lens, nb, bs, budget, sinks, recent)
    assert kvq.kvq_get_device_error() == 0
    assert np.array_equal(kept, np.minimum(lens, budget))
    for b, L in enumerate(lens):
        j = np.arange(L)
        for h in range(hkv):
            want = np.full(budget, -1, np.int32)
            if L <= budget:
                want[:L] = j
            else:
                mid = np.arange(sinks, L - recent)
                w = mass[table[b, mid // bs], h, mid % bs]
                rows = mid[np.lexsort((mid, -w))[:budget - sinks - recent]]
                want[:] = np.sort(np.concatenate([j[:sinks], rows, j[L - recent:]]))
            assert np.array_equal(keep[b, h], want), (b, h)
