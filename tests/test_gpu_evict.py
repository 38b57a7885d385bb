"""The attention weight that keys receive (kvq_key_mass), the rows an eviction
keeps (kvq_evict_select) and their moving (kvq_evict_compact), each against its
64-bit or exact plain form, and all of them run together with the attention."""
import dataclasses

import numpy as np
import pytest
import torch

import score_ref as ref
from guard import guarded
from test_gpu_masked import CASES, check, dev, documents, gpu_cache, run, slopes_of

pytestmark = pytest.mark.gpu

INT8, FP8, INT4 = ref.INT8, ref.FP8, ref.INT4
ROW, TENSOR, CHANNEL, GROUP = ref.ROW, ref.TENSOR, ref.CHANNEL, ref.GROUP


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


# ------------------------------------------------------------------ key mass

def mass_call(kvq, c: ref.Cache, lse, mass, decay=1.0, fresh=None, slopes=None, key_begin=None, key_end=None):
    case = c.case
    g = gpu_cache(kvq, c)
    B = len(case.lens)
    p = kvq.make_params(B, case.hq, case.c, c.width, softcap=case.softcap, window=case.window)
    ws = guarded(torch.zeros(kvq.kvq_key_mass_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda"), "ws")
    m = guarded(dev(mass), "mass")
    f32 = lambda a: None if a is None else dev(np.asarray(a, np.float32))  # noqa: E731
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    mask = kvq.ScoreMask(f32(slopes), i32(key_begin), i32(key_end))
    q, table, lens = dev(c.q).to(torch.bfloat16), dev(c.table), dev(np.array(case.lens, np.int32))
    kvq.kvq_key_mass(g, p, mask, q, table, lens, dev(lse.astype(np.float32)), m, ws, decay=decay, fresh=fresh)
    assert kvq.kvq_get_device_error() == 0
    return m.cpu().numpy()


def random_mass(c: ref.Cache, seed=0):
    r = np.random.default_rng(seed)
    return r.exponential(0.1, (c.nb, c.case.hkv, c.case.bs)).astype(np.float32)


def check_mass(got, c, lse, mass, decay, fresh, slopes=None, key_begin=None, key_end=None):
    want, tol = ref.key_mass(c, lse.astype(np.float32), mass, decay, fresh, slopes, key_begin, key_end)
    untouched = tol == 0
    assert np.array_equal(got[untouched & (want == mass)], mass[untouched & (want == mass)], equal_nan=True)
    worst = (np.abs(got - want) - tol).max()
    assert worst <= 0, f"off by {worst:.2e} more than its bound"


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("c", [1, 4, 8, 11, 30])
def test_mass(kvq, name, c):
    base = CASES[name]
    case = dataclasses.replace(base, c=c, seed=c, lens=tuple(max(L, c) for L in base.lens))
    cache = ref.Cache(case)
    lse = ref.attend(cache)[1]
    mass = random_mass(cache)
    got = mass_call(kvq, cache, lse, mass, decay=0.875)
    check_mass(got, cache, lse, mass, 0.875, c)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 row d256 g6", "fp8 tensor cap", "int4 channel d256",
                                  "latent d576", "int4 group"])
@pytest.mark.parametrize("c", [1, 9, 40])
@pytest.mark.parametrize("decay,fresh", [(1.0, 0), (0.0, 0), (0.5, 3), (1.0, 10 ** 6)])
def test_mass_under_a_rule(kvq, name, c, decay, fresh):
    """Bias, documents, window and empty rows; keys that nobody sees decay."""
    case = dataclasses.replace(CASES[name], c=c, seed=7, lens=(170, max(c, 33)), window=60)
    cache = ref.Cache(case)
    s = slopes_of(case.hq)
    begin, end = documents(case, (25, 101, 150))
    end[0, -1] = 0
    lse = ref.attend(cache, s, begin, end)[1]
    mass = random_mass(cache)
    if decay == 0.0:
        mass[:] = np.nan  # not read
    got = mass_call(kvq, cache, lse, mass, decay, fresh, s, begin, end)
    if decay == 0.0:
        keep = ~np.isnan(got)
        want, tol = ref.key_mass(cache, lse.astype(np.float32), np.zeros_like(mass), 0.0, fresh, s, begin, end)
        for b in range(2):
            blk, row = cache.rows(b)
            assert keep[blk, :, row].all()
            assert (np.abs(got - want)[blk, :, row] <= tol[blk, :, row]).all()
        assert keep.sum() == sum(case.lens) * case.hkv
        return
    check_mass(got, cache, lse, mass, decay, fresh, s, begin, end)


def test_mass_of_a_row_sums_to_one(kvq):
    """Over all keys the weights of each query row add up to one."""
    case = ref.Case(lens=(500, 77), c=6, hq=8, hkv=2)
    cache = ref.Cache(case)
    _, lse = run(kvq, cache)
    got = mass_call(kvq, cache, lse, np.zeros((cache.nb, 2, 16), np.float32))
    for b in range(2):
        blk, row = cache.rows(b)
        # (lse as the attention gave it: 2^-15 and fp32; rows sum G * C)
        assert np.abs(got[blk, :, row].sum(0) - 24).max() <= 24 * 2.0 ** -14


@pytest.mark.parametrize("lens", [(1,), (0, 5), (64,), (65, 63, 1)])
def test_mass_short(kvq, lens):
    case = ref.Case(lens=lens, c=2)
    cache = ref.Cache(case)
    lse = ref.attend(cache)[1]
    mass = random_mass(cache)
    check_mass(mass_call(kvq, cache, lse, mass, 0.5), cache, lse, mass, 0.5, 2)


def test_mass_is_reproducible_and_captured(kvq):
    case = ref.Case(lens=(900, 411), c=24, d=128)
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    lse = dev(ref.attend(cache)[1].astype(np.float32))
    p = kvq.make_params(2, 8, 24, cache.width)
    ws = torch.zeros(kvq.kvq_key_mass_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    q, table, lens = dev(cache.q).to(torch.bfloat16), dev(cache.table), dev(np.array(case.lens, np.int32))
    start = dev(random_mass(cache))
    m1, m2 = start.clone(), start.clone()
    kvq.kvq_key_mass(g, p, None, q, table, lens, lse, m1, ws, decay=0.9)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kvq.kvq_key_mass(g, p, None, q, table, lens, lse, m2, ws, decay=0.9)
    m2.copy_(start)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(m1, m2)


@pytest.mark.parametrize("c", [12, 40])
def test_mass_of_sequences_shorter_than_the_chunk(kvq, c):
    case = ref.Case(lens=(3, 0, 11, 90), c=c, d=128)
    cache = ref.Cache(case)
    s = slopes_of(8)
    lse = ref.attend(cache, s)[1]
    mass = random_mass(cache)
    check_mass(mass_call(kvq, cache, lse, mass, 0.75, slopes=s), cache, lse, mass, 0.75, c, s)


@pytest.mark.parametrize("name", ["int8 row d128", "fp8 row", "int4 group", "int8 row d256 g6", "latent d576"])
@pytest.mark.parametrize("c", [1, 24])
def test_mass_beside_junk(kvq, name, c):
    """Rows that no token sees hold NaN scales and codes: they decay, and
    nothing of them reaches the others."""
    case = dataclasses.replace(CASES[name], c=c, lens=(200,), seed=4)
    cache = ref.Cache(case)
    begin = np.full((1, c), 70, np.int32)
    end = np.full((1, c), 150, np.int32)
    lse = ref.attend(cache, None, begin, end)[1]
    mass = random_mass(cache)
    want, tol = ref.key_mass(cache, lse.astype(np.float32), mass, 0.5, 0, None, begin, end)
    blk, row = cache.rows(0)
    bad = np.r_[0:70, 150:200]
    if case.dtype == FP8:
        cache.k_codes[blk[bad], :, row[bad]] = 0x7F
    if cache.k_scale.ndim >= 3:
        cache.k_scale[blk[bad], :, row[bad]] = np.nan
    got = mass_call(kvq, cache, lse, mass, 0.5, 0, None, begin, end)
    assert (np.abs(got - want)[blk, :, row] <= tol[blk, :, row]).all()


@pytest.mark.parametrize("hq,hkv,c", [(7, 1, 3), (10, 2, 30), (9, 3, 50), (8, 1, 16), (8, 1, 17), (6, 1, 22)])
def test_mass_group_sizes(kvq, hq, hkv, c):
    """Row counts around the kernels' tiles (8, 16, 32, 64, 128 rows), one launch
    and several, with and without the tensor-memory kernel."""
    for d, km in ((128, ROW), (256, CHANNEL), (64, TENSOR)):
        case = ref.Case(d=d, km=km, vm=km, hq=hq, hkv=hkv, c=c, lens=(300, 77), seed=hq)
        cache = ref.Cache(case)
        s = slopes_of(hq, -0.02)
        lse = ref.attend(cache, s)[1]
        mass = random_mass(cache)
        check_mass(mass_call(kvq, cache, lse, mass, 0.9, slopes=s), cache, lse, mass, 0.9, c, s)


# -------------------------------------------------------------------- select

def pages(lens, bs, seed, slack=2, width=None):
    r = np.random.default_rng(seed)
    need = [max(1, -(-L // bs)) for L in lens]
    nb = sum(need) + slack
    perm = r.permutation(nb).astype(np.int32)
    table = np.full((len(lens), width or max(need)), nb - 1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, nb


def select_call(kvq, mass, table, lens, nb, bs, budget, sinks, recent, max_seq_len=0):
    hkv = mass.shape[1]
    p = kvq.make_evict_params(len(lens), table.shape[1], budget, num_blocks=nb, block_size=bs, num_kv_heads=hkv,
                              sinks=sinks, recent=recent, max_seq_len=max_seq_len)
    keep = guarded(torch.full((len(lens), hkv, budget), -9, dtype=torch.int32, device="cuda"), "keep")
    kept = guarded(torch.full((len(lens),), -9, dtype=torch.int32, device="cuda"), "kept")
    kvq.kvq_evict_select(p, dev(mass), dev(table), dev(np.array(lens, np.int32)), keep, kept)
    return keep.cpu().numpy(), kept.cpu().numpy()


def check_select(kvq, mass, lens, bs, budget, sinks, recent, seed=0, width=None, **kw):
    table, nb = pages(lens, bs, seed, width=width)
    full = mass(nb)
    got = select_call(kvq, full, table, lens, nb, bs, budget, sinks, recent, **kw)
    assert kvq.kvq_get_device_error() == 0
    want = ref.select(full, table, lens, bs, budget, sinks, recent)
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])


def masses(kind, hkv, bs, seed=0):
    r = np.random.default_rng(seed)

    def make(nb):
        shape = (nb, hkv, bs)
        if kind == "weights":
            return r.exponential(0.01, shape).astype(np.float32)
        if kind == "equal":
            return np.full(shape, 0.25, np.float32)
        if kind == "few":
            return r.integers(0, 3, shape).astype(np.float32)
        if kind == "close":  # differ in the last bits only
            return (np.float32(1.0).view(np.uint32) + r.integers(0, 5, shape)).astype(np.uint32).view(np.float32)
        x = r.standard_normal(shape).astype(np.float32)  # odd: both signs, zeros, infinities, NaN
        x[r.random(shape) < 0.2] = 0.0
        x[r.random(shape) < 0.2] = -0.0
        x[r.random(shape) < 0.1] = np.nan
        x[r.random(shape) < 0.05] = -np.nan
        x[r.random(shape) < 0.05] = np.inf
        x[r.random(shape) < 0.05] = -np.inf
        x[r.random(shape) < 0.05] = 1e-42
        return x
    return make


@pytest.mark.parametrize("kind", ["weights", "equal", "few", "close", "odd"])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ((300,), 100, 4, 16), ((17, 16, 15, 0, 1), 16, 2, 3), ((5000, 2048, 33), 777, 0, 0), ((1000,), 999, 1, 0),
    ((1000,), 20, 10, 10), ((4097,), 1, 0, 0), ((4097,), 1, 0, 1), ((9000, 8999), 4096, 4, 512),
])
def test_select(kvq, kind, lens, budget, sinks, recent):
    check_select(kvq, masses(kind, 3, 16), lens, 16, budget, sinks, recent)


@pytest.mark.parametrize("near", [1, 2, 511, 513, 1025, 2047, 2048, 2049, 6000])
@pytest.mark.parametrize("kinds", [1, 7, 1 << 16])
@pytest.mark.parametrize("neg", [False, True])
def test_select_among_weights_of_one_upper_half(kvq, near, kinds, neg):
    """`near` weights share the threshold's upper 16 bits (and take `kinds` lower
    halves), with others above and below: around the number that is sorted out
    on chip, over several CTAs, the threshold at either end and in the middle."""
    r = np.random.default_rng(near + kinds)
    L = 9000
    table, nb = pages((L,), 64, 3)
    up, down = (L - near) // 3, L - near - (L - near) // 3
    w = np.concatenate([r.uniform(2.0, 9.0, up), r.uniform(0.0, 0.9, down)]).astype(np.float32)
    low = (r.integers(0, kinds, near) * (65535 // max(1, kinds - 1) if kinds > 1 else 1)).astype(np.uint32)
    w = np.concatenate([w, (np.uint32(0x3F800000) + low).view(np.float32)])
    w = r.permutation(-w if neg else w)
    mass = np.zeros((nb, 1, 64), np.float32)
    j = np.arange(L)
    mass[table[0, j // 64], 0, j % 64] = w
    above = down if neg else up
    for budget in sorted({above + 1, above + (near + 1) // 2, above + near}):
        got = select_call(kvq, mass, table, (L,), nb, 64, budget, 0, 0)
        want = ref.select(mass, table, (L,), 64, budget, 0, 0)
        assert np.array_equal(got[0], want[0])
    assert kvq.kvq_get_device_error() == 0


MANY = (20000, 12001, 9000, 8300, 8193, 4097, 3000, 2047, 1024, 777, 512, 300, 100, 65, 64, 33, 31, 1, 0)


@pytest.mark.parametrize("kind", ["weights", "equal", "few", "close", "odd"])
@pytest.mark.parametrize("bs,budget,sinks,recent", [(16, 700, 4, 16), (64, 64, 0, 0), (256, 6000, 33, 500),
                                                    (1024, 8192, 1, 0), (32, 40, 3, 36)])
def test_select_of_many_heads(kvq, kind, bs, budget, sinks, recent):
    """A head or more per SM (152 here) of up to 40,960 rows: one pass between
    sampled bounds, and the digits over all rows where the weights are too alike
    for it."""
    check_select(kvq, masses(kind, 8, bs), MANY, bs, budget, sinks, recent, width=40960 // bs)


@pytest.mark.parametrize("what", ["sample", "ties", "steps", "tail"])
def test_select_of_many_heads_against_the_sample(kvq, what):
    """Weights that the evenly spread sample tells nothing about: other values
    at the sampled rows, one value almost everywhere, a few values, and every
    large weight in one stretch."""
    r = np.random.default_rng(5)
    lens, bs, hkv, budget = (20000,) * 4, 64, 40, 5000
    table, nb = pages(lens, bs, 1, width=640)
    mass = np.zeros((nb, hkv, bs), np.float32)
    j = np.arange(20000)
    for b in range(4):
        for h in range(hkv):
            w = r.exponential(1.0, 20000).astype(np.float32)
            if what == "sample":
                w[(np.arange(4096) * 20000) >> 12] = 1e6 if h % 2 else 1e-6
            elif what == "ties":
                w[r.random(20000) < 0.97] = 0.5 if h % 2 else 0.0
            elif what == "steps":
                w = np.floor(4.0 * w).astype(np.float32)
            else:
                w[: 20000 - budget - (h - 20) * 40] *= 1e-3
            mass[table[b, j // bs], h, j % bs] = w
    got = select_call(kvq, mass, table, lens, nb, bs, budget, 0, 0)
    assert kvq.kvq_get_device_error() == 0
    for b in range(4):
        for h in range(hkv):
            w = mass[table[b, j // bs], h, j % bs]
            want = np.sort(np.lexsort((j, -w))[:budget])  # the largest, ties to the lower row
            assert np.array_equal(got[0][b, h], want), (b, h)


def test_select_long_and_wide(kvq):
    """Sixteen CTAs to a head; a part longer than the keys a CTA keeps on chip
    (read again from global memory); lengths far below the bound."""
    check_select(kvq, masses("weights", 1, 256), (70001,), 256, 20000, 4, 1000)
    check_select(kvq, masses("few", 2, 256), (262144,), 256, 65536, 4, 8192)
    check_select(kvq, masses("few", 1, 1024), (900_000, 5, 900_001), 1024, 450_000, 4, 1)
    check_select(kvq, masses("weights", 8, 64), tuple(range(1, 3000, 61)), 64, 64, 4, 8)


def test_select_flags(kvq):
    table, nb = pages((100, 100), 16, 1)
    m = masses("weights", 2, 16)(nb)
    select_call(kvq, m, table, (100, 10 ** 6), nb, 16, 32, 0, 0)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SEQ_LEN
    bad = table.copy()
    bad[0, 2] = -1
    got, _ = select_call(kvq, m, bad, (100, 100), nb, 16, 32, 0, 0)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_ID
    assert not np.isin(got[0], np.arange(32, 48)).any()  # its rows rank last


# ------------------------------------------------------------------- compact

def compact_call(kvq, c: ref.Cache, keep, kept, mass, dst=None):
    case = c.case
    g = gpu_cache(kvq, c)
    p = kvq.make_evict_params(len(case.lens), c.width, keep.shape[2], num_blocks=c.nb, block_size=case.bs,
                              num_kv_heads=case.hkv)
    ws = guarded(torch.full((kvq.kvq_evict_compact_workspace_size(g, p) // 4,), 7, dtype=torch.int32, device="cuda"),
                 "ws")
    m = None if mass is None else guarded(dev(mass), "mass")
    kvq.kvq_evict_compact(g, p, dev(c.table), None if dst is None else dev(dst), dev(keep), dev(kept), m, ws)
    assert kvq.kvq_get_device_error() == 0
    return g, m


def check_compact(kvq, case, budget, seed=0, out_of_place=False, with_mass=True):
    cache = ref.Cache(case)
    r = np.random.default_rng(seed)
    keep = np.full((len(case.lens), case.hkv, budget), -1, np.int32)
    kept = np.minimum(case.lens, budget).astype(np.int32)
    for b, L in enumerate(case.lens):
        for h in range(case.hkv):
            keep[b, h, :kept[b]] = np.sort(r.permutation(L)[:kept[b]])
    mass = random_mass(cache) if with_mass else None
    dst = cache.table
    if out_of_place:
        need = -(-budget // case.bs)
        free = np.setdiff1d(np.arange(cache.nb), np.unique(cache.table))
        assert len(free) >= need * len(case.lens)
        dst = np.full_like(cache.table, -1)  # entries behind the kept rows are not read
        dst[:, :need] = free[:need * len(case.lens)].reshape(len(case.lens), need)
    g, m = compact_call(kvq, cache, keep, kept, mass, dst if out_of_place else None)
    arrays = [cache.k_codes] + ([] if case.latent else [cache.v_codes])
    names = ["k_codes"] + ([] if case.latent else ["v_codes"])
    for side, mode in (("k", case.km), ("v", case.vm)):
        if mode in (ROW, GROUP) and not (side == "v" and case.latent):
            arrays.append(getattr(cache, side + "_scale"))
            names.append(side + "_scale")
    if with_mass:
        arrays.append(mass)
        names.append("mass")
    want = ref.compact(arrays, cache.table, dst, keep, kept, case.bs)
    for name, w in zip(names, want):
        got = m.cpu().numpy() if name == "mass" else getattr(g, name).cpu().numpy()
        assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(w).view(np.uint8)), name


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("lens,budget", [((333, 100, 1), 60), ((200, 128), 128), ((64, 0, 63), 64), ((700,), 1)])
def test_compact_in_place(kvq, name, lens, budget):
    check_compact(kvq, dataclasses.replace(CASES[name], lens=lens), budget)


@pytest.mark.parametrize("name", ["int8 row d128", "int4 group", "fp8 tensor cap", "latent d576"])
@pytest.mark.parametrize("bs", [16, 128])
def test_compact_out_of_place(kvq, name, bs):
    check_compact(kvq, dataclasses.replace(CASES[name], lens=(333, 100, 1), bs=bs, slack=20), 90, out_of_place=True)


@pytest.mark.parametrize("bs,d", [(16, 64), (256, 256), (1024, 128)])
def test_compact_many_rounds(kvq, bs, d):
    """Enough rows that every block takes several units of each head, most of
    them reading rows that other blocks overwrite."""
    check_compact(kvq, ref.Case(d=d, lens=(30011, 17000), bs=bs, hkv=4, hq=4), 16384, seed=bs)


def test_compact_without_weights(kvq):
    check_compact(kvq, ref.Case(lens=(500, 90)), 77, with_mass=False)


def test_compact_bad_index_is_flagged(kvq):
    case = ref.Case(lens=(100,))
    cache = ref.Cache(case)
    keep = np.sort(np.random.default_rng(1).permutation(100)[:20]).astype(np.int32)
    keep = np.broadcast_to(keep, (1, 2, 20)).copy()
    for bad in (-1, 10 ** 6):
        k = keep.copy()
        k[0, 1, 7] = bad
        g = gpu_cache(kvq, cache)
        p = kvq.make_evict_params(1, cache.width, 20, num_blocks=cache.nb, block_size=16, num_kv_heads=2)
        ws = torch.zeros(kvq.kvq_evict_compact_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
        kvq.kvq_evict_compact(g, p, dev(cache.table), None, dev(k), dev(np.array([20], np.int32)), None, ws)
        assert kvq.kvq_get_device_error() == kvq.DEVERR_KEEP_INDEX
        # the other head's rows arrived
        want = ref.compact([cache.k_codes], cache.table, cache.table, keep, np.array([20]), 16)[0]
        i = np.arange(20)
        got = g.k_codes.cpu().numpy()
        assert np.array_equal(got[cache.table[0, i // 16], 0, i % 16], want[cache.table[0, i // 16], 0, i % 16])


def test_compact_is_captured(kvq):
    """A captured in-place move, replayed on restored contents."""
    case = ref.Case(lens=(5000, 3000), d=128, hkv=4, hq=4)
    cache = ref.Cache(case)
    r = np.random.default_rng(3)
    keep = np.stack([[np.sort(r.permutation(L)[:1500]) for _ in range(4)] for L in case.lens]).astype(np.int32)
    g = gpu_cache(kvq, cache)
    k0 = g.k_codes.clone()
    p = kvq.make_evict_params(2, cache.width, 1500, num_blocks=cache.nb, block_size=16, num_kv_heads=4)
    ws = torch.zeros(kvq.kvq_evict_compact_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    table, kd, n = dev(cache.table), dev(keep), dev(np.array([1500, 1500], np.int32))
    kvq.kvq_evict_compact(g, p, table, None, kd, n, None, ws)
    torch.cuda.synchronize()
    want = g.k_codes.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kvq.kvq_evict_compact(g, p, table, None, kd, n, None, ws)
    for _ in range(3):
        g.k_codes.copy_(k0)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(g.k_codes, want)
    assert kvq.kvq_get_device_error() == 0


# ----------------------------------------------------- caches beyond 4 GB

def test_pages_beyond_four_gigabytes(kvq):
    """The same rows in pages behind the first 4 GB of a 5 GB pool and in a small
    pool: attention, weights, selection and moves agree bit for bit."""
    nb, bs, hkv, d, far = 20480, 256, 8, 128, 20000
    L, n_pages, budget = 1500, 6, 600
    r = np.random.default_rng(1)
    small = kvq.QuantizedPagedCache(INT8, ROW, ROW, 8, bs, hkv, d)
    big = kvq.QuantizedPagedCache(INT8, ROW, ROW, nb, bs, hkv, d)
    assert big.k_codes[:far].numel() > 4 << 30
    kv = [torch.from_numpy(r.standard_normal((L, hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in "kv"]
    order = r.permutation(n_pages).astype(np.int32)
    outs = []
    for g, first in ((small, 0), (big, far)):
        pages = order + first
        slots = pages[np.arange(L) // bs].astype(np.int64) * bs + np.arange(L) % bs
        kvq.kvq_append(g, kv[0], kv[1], dev(slots))
        table = dev(pages[None])
        lens = dev(np.array([L], np.int32))
        res = []
        for c in (1, 40):
            p = kvq.make_params(1, 16, c, n_pages)
            q = torch.from_numpy(np.random.default_rng(c).standard_normal((1, c, 16, d)).astype(np.float32))
            q = q.to(torch.bfloat16).cuda()
            ws = torch.zeros(max(kvq.kvq_attend_masked_workspace_size(g, p), kvq.kvq_key_mass_workspace_size(g, p)) // 4,
                             dtype=torch.int32, device="cuda")
            out = torch.zeros((1, c, 16, d), dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros((1, c, 16), device="cuda")
            rule = kvq.ScoreMask(slopes=dev(np.array(slopes_of(16), np.float32)))
            kvq.kvq_attend_masked(g, p, rule, q, table, lens, None, out, lse, ws)
            mass = torch.zeros((g.num_blocks, hkv, bs), device="cuda")
            kvq.kvq_key_mass(g, p, rule, q, table, lens, lse, mass, ws)
            res += [out, lse, mass[first:first + n_pages].clone()]
        ep = kvq.make_evict_params(1, n_pages, budget, num_blocks=g.num_blocks, block_size=bs, num_kv_heads=hkv,
                                   recent=50)
        b = kvq.alloc_evict_buffers(g, ep)
        kvq.evict_step(g, ep, table, lens, mass, b)
        res += [b.keep, b.kept_lens, mass[first:first + n_pages].clone()]
        res += [t[first:first + n_pages].clone() for t in (g.k_codes, g.v_codes, g.k_scale, g.v_scale)]
        outs.append(res)
    assert kvq.kvq_get_device_error() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("steps", [6])
def test_decode_with_evictions(kvq, steps):
    """Steps as a server runs them: append, attention under a bias, weights,
    and an eviction whenever a sequence outgrows its budget; each step's
    output against the 64-bit attention over the rows that are there."""
    hq, hkv, d, bs, budget, cap = 8, 2, 128, 16, 48, 64
    B, nb, width = 2, 10, 4
    r = np.random.default_rng(0)
    table = r.permutation(nb)[:B * width].reshape(B, width).astype(np.int32)
    g = kvq.QuantizedPagedCache(INT8, ROW, ROW, nb, bs, hkv, d)
    mass = torch.zeros((nb, hkv, bs), device="cuda")
    slopes = dev(np.array(slopes_of(hq), np.float32))
    tbl = dev(table)
    lens = np.array([40, 57], np.int32)
    ep = kvq.make_evict_params(B, width, budget, num_blocks=nb, block_size=bs, num_kv_heads=hkv, sinks=2, recent=8)
    eb = kvq.alloc_evict_buffers(g, ep)

    def append(counts):
        k, v, s = [], [], []
        for b in range(B):
            for p in range(int(lens[b]) - counts, int(lens[b])):
                s.append(table[b, p // bs] * bs + p % bs)
        n = len(s)
        k, v = (torch.from_numpy(ref.bf16(r.standard_normal((n, hkv, d)))).to(torch.bfloat16).cuda() for _ in "kv")
        kvq.kvq_append(g, k, v, dev(np.array(s, np.int64)))

    # the history, as one chunk of 40 tokens each
    append(40)
    evicted = 0
    for step in range(steps):
        c = 40 if step == 0 else 3
        if step > 0:
            lens = lens + 3
            append(3)
        case = ref.Case(d=d, hq=hq, hkv=hkv, bs=bs, lens=tuple(int(x) for x in lens), c=c)
        cache = ref.Cache(case, width=width)
        cache.nb, cache.table = nb, table
        cache.q = ref.bf16(r.standard_normal((B, c, hq, d)))
        p = kvq.make_params(B, hq, c, width)
        n = max(kvq.kvq_attend_masked_workspace_size(g, p), kvq.kvq_key_mass_workspace_size(g, p))
        ws = torch.zeros(n // 4, dtype=torch.int32, device="cuda")
        out = torch.zeros((B, c, hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((B, c, hq), device="cuda")
        rule = kvq.ScoreMask(slopes=slopes)
        q, ld = dev(cache.q).to(torch.bfloat16), dev(lens)
        before = mass.cpu().numpy()
        cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale = (
            t.cpu().numpy() for t in (g.k_codes, g.v_codes, g.k_scale, g.v_scale))
        kvq.kvq_attend_masked(g, p, rule, q, tbl, ld, None, out, lse, ws)
        kvq.kvq_key_mass(g, p, rule, q, tbl, ld, lse, mass, ws, decay=0.5)
        s = slopes_of(hq)
        check(cache, (out.double().cpu().numpy(), lse.double().cpu().numpy()), s)
        check_mass(mass.cpu().numpy(), cache, lse.cpu().numpy(), before, 0.5, c, s)
        if (lens > budget).any():
            want, new = ref.select(mass.cpu().numpy(), table, [int(x) for x in lens], bs, budget, 2, 8)
            arrays = [t.cpu().numpy() for t in (g.k_codes, g.v_codes, g.k_scale, g.v_scale, mass)]
            moved = ref.compact(arrays, table, table, want, new, bs)
            kept = kvq.evict_step(g, ep, tbl, ld, mass, eb)
            assert np.array_equal(eb.keep.cpu().numpy(), want)
            for t, w in zip((g.k_codes, g.v_codes, g.k_scale, g.v_scale, mass), moved):
                assert np.array_equal(t.cpu().numpy(), w)
            lens = kept.cpu().numpy()
            evicted += 1
    assert evicted >= 2 and cap >= budget
    assert kvq.kvq_get_device_error() == 0


def test_refuses_wrong_tensors(kvq):
    case = ref.Case(lens=(50,), c=2)
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(1, 8, 2, cache.width)
    ws = torch.zeros(4096, dtype=torch.int32, device="cuda")
    q, table, lens = dev(cache.q).to(torch.bfloat16), dev(cache.table), dev(np.array([50], np.int32))
    lse, mass = torch.zeros((1, 2, 8), device="cuda"), torch.zeros((cache.nb, 2, 16), device="cuda")
    for a in ((q, table, lens, lse.double(), mass), (q, table, lens, lse, mass[1:]), (q[:, :1], table, lens, lse, mass),
              (q, table, lens, lse, mass.transpose(1, 2))):
        with pytest.raises(ValueError):
            kvq.kvq_key_mass(g, p, None, *a, ws)
    for kw in (dict(decay=1.5), dict(decay=-0.1), dict(decay=float("nan")), dict(fresh=-1)):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_key_mass(g, p, None, q, table, lens, lse, mass, ws, **kw)
    ep = kvq.make_evict_params(1, cache.width, 20, num_blocks=cache.nb, block_size=16, num_kv_heads=2)
    keep = torch.zeros((1, 2, 20), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        kvq.kvq_evict_select(ep, mass, table, lens, keep[:, :1], lens.clone())
    with pytest.raises(kvq.KvqError):
        kvq.kvq_evict_select(ep, mass, table, lens, keep, lens)  # lengths in and out are one tensor
    other = kvq.make_evict_params(1, cache.width, 20, num_blocks=cache.nb + 1, block_size=16, num_kv_heads=2)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_evict_compact(g, other, table, None, keep, lens.clone(), None, ws)


# ------------------------------------------------- padding with odd contents

@pytest.mark.parametrize("name", ["int8 row d128", "fp8 tensor cap", "int4 channel d256", "int8 row d256 g6",
                                  "int8 channel d64", "int8 group k, row v", "latent d576"])
@pytest.mark.parametrize("c", [1, 3, 12, 40, 130])
@pytest.mark.parametrize("junk", [np.nan, np.inf])
def test_padding_tokens_may_hold_anything(kvq, name, c, junk):
    """A padded batch: the queries of tokens that see nothing hold NaN or
    infinities, which reach neither the other tokens' rows nor the keys."""
    case = dataclasses.replace(CASES[name], c=c, seed=c, lens=(max(c, 333), max(c, 150), 150 + c))
    cache = ref.Cache(case)
    s = slopes_of(case.hq)
    end = np.stack([L - c + np.arange(c) + 1 for L in case.lens]).astype(np.int32)
    end[0, ::2] = 0         # every second token
    end[1] = -1             # a whole sequence
    end[2, c // 2:] = 5     # the tail, by an interval that ends before it begins
    begin = np.zeros_like(end)
    begin[2, c // 2:] = 9
    r_lse = ref.attend(cache, s, begin, end)[1]
    mass = random_mass(cache)
    clean = cache.q.copy()
    dead = end <= begin
    cache.q[dead] = junk
    cache.q[dead, :, ::3] = 1.0
    got = run(kvq, cache, s, begin, end)
    m = mass_call(kvq, cache, r_lse, mass, 0.5, c, s, begin, end)
    cache.q = clean  # the plain forms see the queries without the junk
    check(cache, got, s, begin, end)
    check_mass(m, cache, r_lse, mass, 0.5, c, s, begin, end)


@pytest.mark.parametrize("last,err", [(59, 0), (18, 1), (0, 1)])
def test_compact_refuses_rows_from_before(kvq, last, err):
    """In place a kept row from before its destination (here row 19's) is flagged
    and not moved; the same row twice is copied twice."""
    case = ref.Case(lens=(100,), hkv=1, hq=4)
    cache = ref.Cache(case)
    keep = np.arange(40, 60).astype(np.int32).reshape(1, 1, 20)
    keep[0, 0, 4] = keep[0, 0, 3]
    keep[0, 0, 19] = last
    g = gpu_cache(kvq, cache)
    p = kvq.make_evict_params(1, cache.width, 20, num_blocks=cache.nb, block_size=16, num_kv_heads=1)
    ws = torch.zeros(kvq.kvq_evict_compact_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    kvq.kvq_evict_compact(g, p, dev(cache.table), None, dev(keep), dev(np.array([20], np.int32)), None, ws)
    assert kvq.kvq_get_device_error() == (kvq.DEVERR_KEEP_INDEX if err else 0)
    got = g.k_codes.cpu().numpy()
    for i in range(19 if err else 20):
        src = keep[0, 0, i]
        assert np.array_equal(got[cache.table[0, i // 16], 0, i % 16],
                              cache.k_codes[cache.table[0, src // 16], 0, src % 16])


def test_select_of_many_heads_bad_pages_alignment_and_capture(kvq):
    """A page outside the pool is flagged and its rows rank last; weights at an
    address that 16-byte loads cannot take give the same rows, as do a call on
    another stream and a replayed one."""
    r = np.random.default_rng(9)
    B, hkv, bs, L, budget = 20, 8, 64, 33000, 900
    table, nb = pages((L,) * B, bs, 2)
    w = r.exponential(1.0, (nb, hkv, bs)).astype(np.float32)
    p = kvq.make_evict_params(B, table.shape[1], budget, num_blocks=nb, block_size=bs, num_kv_heads=hkv, sinks=5,
                              recent=40)
    lens, tbl = dev(np.full(B, L, np.int32)), dev(table)
    aligned = dev(w)
    shifted = torch.zeros(w.size + 1, device="cuda")[1:].view(w.shape)
    shifted.copy_(aligned)
    keep = torch.full((B, hkv, budget), -9, dtype=torch.int32, device="cuda")
    kept = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    kvq.kvq_evict_select(p, aligned, tbl, lens, keep, kept)
    j = np.arange(L)
    for b, h in ((0, 0), (7, 3), (19, 7)):
        v = w[table[b, j // bs], h, j % bs]
        mid = 5 + np.lexsort((j[5:-40], -v[5:-40]))[:budget - 45]
        want = np.concatenate([np.arange(5), np.sort(mid), np.arange(L - 40, L)])
        assert np.array_equal(keep[b, h].cpu().numpy(), want)
    assert (kept == budget).all()
    other = torch.zeros_like(keep)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvq.kvq_evict_select(p, aligned, tbl, lens, other, kept, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(keep, other)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kvq.kvq_evict_select(p, aligned, tbl, lens, other, kept)
    other.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(keep, other)
    kvq.kvq_evict_select(p, shifted, tbl, lens, other, kept)
    assert torch.equal(keep, other)
    assert kvq.kvq_get_device_error() == 0
    # two pages of sequence 3, one outside the pool on either side
    bad = table.copy()
    bad[3, 100], bad[3, 200] = nb, -1
    kvq.kvq_evict_select(p, aligned, dev(bad), lens, other, kept)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_ID
    same = [b for b in range(B) if b != 3]
    assert torch.equal(keep[same], other[same])
    at = other[3].cpu().numpy() // bs
    assert not np.isin(at, (100, 200)).any()
