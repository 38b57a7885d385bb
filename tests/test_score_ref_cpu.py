"""The plain forms the GPU tests compare with, on the CPU: against torch's own
operations and the oracle, and with planted mistakes; and the argument checks
of the entry points, which run before any CUDA call."""
import ctypes

import numpy as np
import pytest

import score_ref as ref

FAKE = 0x7F0000000000  # an aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import build, kvq
    build.build()
    kvq.load()
    return kvq


def test_attend_matches_the_oracle(orc):
    """Causal with a window, cap and sink: the same rows as the oracle's."""
    case = ref.Case(lens=(50, 33), c=3, softcap=20.0, window=17)
    c = ref.Cache(case)
    oc = orc.OracleCache(1, 1, 1, c.nb, case.bs, case.hkv, case.d)
    oc.k_codes[:], oc.v_codes[:] = c.k_codes, c.v_codes
    oc.k_scale[:], oc.v_scale[:] = c.k_scale, c.v_scale
    sink = np.linspace(-1, 1, 8).astype(np.float32)
    q = (c.q.view(np.uint32) >> 16).astype(np.uint16)
    want, lse = oc.attend(q, c.table, np.array(case.lens, np.int32), q_tokens=3, softcap=20.0, window=17,
                          head_sink=sink)
    out, l, *_ = ref.attend(c, sink=sink)
    assert np.allclose(out, want, rtol=1e-6, atol=1e-7) and np.allclose(l, lse, rtol=1e-6)


def test_rules_of_one_row():
    """Bias and interval of a single row against the formula written out."""
    case = ref.Case(lens=(9,), c=1, hq=1, hkv=1, d=64)
    c = ref.Cache(case)
    out, lse, *_ = ref.attend(c, slopes=[0.5], key_begin=np.array([[2]]), key_end=np.array([[7]]))
    k, v, q = c.values(0, 0, "k"), c.values(0, 0, "v"), c.q[0, 0, 0].astype(float)
    s = np.array([k[j] @ q / 8 - 0.5 * (8 - j) for j in range(2, 7)])
    assert np.isclose(lse[0, 0, 0], np.log(np.exp(s).sum()))
    assert np.allclose(out[0, 0, 0], np.exp(s - lse[0, 0, 0]) @ v[2:7])


def test_mass_rows_sum_to_one_and_mistakes_show():
    case = ref.Case(lens=(40,), c=4)
    c = ref.Cache(case)
    lse = ref.attend(c)[1]
    zero = np.zeros((c.nb, 2, 16), np.float32)
    new, tol = ref.key_mass(c, lse, zero, 1.0, 0)
    assert np.allclose(new.sum((0, 2)), 4 * 4)
    wrong, _ = ref.key_mass(c, lse + 1e-3, zero, 1.0, 0)
    assert (np.abs(wrong - new) > tol).sum() > 70  # a log-sum-exp off by 1e-3 is out of bounds


def test_select_and_compact_by_hand():
    m = np.zeros((2, 1, 16), np.float32)
    m[0, 0, :6] = [1, np.nan, 3, -0.0, 0.0, 2]
    keep, n = ref.select(m, np.array([[0, 1]], np.int32), [6], 16, 4, 0, 0)
    assert keep.tolist() == [[[0, 2, 3, 5]]] and n.tolist() == [4]
    keep, n = ref.select(m, np.array([[0, 1]], np.int32), [6], 16, 4, 2, 1)
    assert keep.tolist() == [[[0, 1, 2, 5]]]
    a = np.arange(32).reshape(2, 1, 16)
    t = np.array([[1, 0]])
    assert ref.compact([a], t, t, keep, n, 16)[0][1, 0, :6].tolist() == [16, 17, 18, 21, 20, 21]


def cache_desc(kvq, **kw):
    d = dict(dtype=1, k_mode=1, v_mode=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, k_codes=FAKE,
             v_codes=FAKE + 4096, k_scale=FAKE + 8192, v_scale=FAKE + 16384)
    d.update(kw)
    return kvq.CacheDesc(**d)


def params(kvq, **kw):
    d = dict(batch=2, num_q_heads=8, q_tokens=5, max_blocks_per_seq=4)
    d.update(kw)
    return kvq.DecodeParams(**d)


BAD_PARAMS = [
    (dict(q_tokens=0), 1), (dict(num_q_heads=7), 1), (dict(num_q_heads=0), 1), (dict(num_q_heads=18), 2),
    (dict(batch=-1), 1), (dict(batch=1025), 2), (dict(max_blocks_per_seq=0), 1), (dict(window=-1), 1),
    (dict(softcap=-1.0), 1), (dict(sm_scale=float("nan")), 1), (dict(batch=1024, q_tokens=2 ** 30), 2),
    (dict(max_blocks_per_seq=2 ** 28), 1),
]


@pytest.mark.parametrize("bad,status", BAD_PARAMS)
def test_masked_and_mass_refuse_params(kvq, bad, status):
    lib, c, p = kvq.load(), cache_desc(kvq), params(kvq, **bad)
    n = ctypes.c_size_t(0)
    a = [ctypes.byref(c), ctypes.byref(p)]
    assert lib.kvq_attend_masked(*a, None, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, 1 << 40, None) == status
    assert lib.kvq_key_mass(*a, None, FAKE, FAKE, FAKE, FAKE, 1.0, 0, FAKE, FAKE, 1 << 40, None) == status
    assert lib.kvq_attend_masked_workspace_size(*a, ctypes.byref(n)) == status
    assert lib.kvq_key_mass_workspace_size(*a, ctypes.byref(n)) == status


def test_masked_and_mass_refuse_pointers(kvq):
    lib, c, p = kvq.load(), cache_desc(kvq), params(kvq)
    good = dict(mask=None, q=FAKE, table=FAKE, lens=FAKE, sink=None, out=FAKE, lse=None, ws=FAKE)

    def attend(**kw):
        v = {**good, **kw}
        return lib.kvq_attend_masked(ctypes.byref(c), ctypes.byref(p), v["mask"], v["q"], v["table"], v["lens"],
                                     v["sink"], v["out"], v["lse"], v["ws"], 1 << 40, None)

    def mass(decay=1.0, fresh=0, **kw):
        v = {**good, "lse": FAKE, **kw}
        return lib.kvq_key_mass(ctypes.byref(c), ctypes.byref(p), v["mask"], v["q"], v["table"], v["lens"], v["lse"],
                                decay, fresh, v["out"], v["ws"], 1 << 40, None)

    for f in (attend, mass):
        for kw in (dict(q=None), dict(q=FAKE + 8), dict(table=None), dict(table=FAKE + 2), dict(lens=None),
                   dict(out=None), dict(ws=None), dict(ws=FAKE + 128), dict(lse=FAKE + 1)):
            assert f(**kw) == 1, kw
        for field in ("slopes", "key_begin", "key_end"):
            m = kvq.ScoreMaskDesc(**{field: FAKE + 2})
            assert f(mask=ctypes.byref(m)) == 1
    assert attend(out=FAKE + 8) == 1 and attend(sink=FAKE + 2) == 1
    for d in (-0.5, 1.5, float("nan"), float("inf")):
        assert mass(decay=d) == 1
    assert mass(fresh=-1) == 1
    assert lib.kvq_attend_masked(None, ctypes.byref(p), None, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, 1, None) == 1
    assert lib.kvq_attend_masked(ctypes.byref(c), None, None, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, 1, None) == 1


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(max_blocks_per_seq=0), dict(num_blocks=0), dict(block_size=24), dict(block_size=8),
    dict(num_kv_heads=0), dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13),
    dict(budget=65), dict(max_seq_len=-1), dict(max_blocks_per_seq=2 ** 28),
])
def test_evict_refuses_params(kvq, bad):
    d = dict(batch=2, max_blocks_per_seq=4, max_seq_len=0, num_blocks=8, block_size=16, num_kv_heads=2, budget=32,
             sinks=0, recent=0)
    d.update(bad)
    lib, c, p = kvq.load(), cache_desc(kvq), kvq.EvictParams(**d)
    n = ctypes.c_size_t(0)
    assert lib.kvq_evict_select(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE, FAKE + 4, None) == 1
    assert lib.kvq_evict_compact(ctypes.byref(c), ctypes.byref(p), FAKE, None, FAKE, FAKE, None, FAKE, 1 << 40,
                                 None) == 1
    assert lib.kvq_evict_compact_workspace_size(ctypes.byref(c), ctypes.byref(p), ctypes.byref(n)) == 1


def test_evict_refuses_pointers(kvq):
    lib, c = kvq.load(), cache_desc(kvq)
    p = kvq.make_evict_params(2, 4, 32, num_blocks=8, block_size=16, num_kv_heads=2)
    s = [FAKE, FAKE, FAKE, FAKE, FAKE + 4]
    for i in range(5):
        for bad in (None, FAKE + 2):
            a = list(s)
            a[i] = bad
            assert lib.kvq_evict_select(ctypes.byref(p), *a, None) == 1
    assert lib.kvq_evict_select(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE, FAKE, None) == 1  # lengths in = out
    m = [FAKE, None, FAKE, FAKE, None, FAKE]
    for i, bads in ((0, (None, FAKE + 2)), (1, (FAKE + 2,)), (2, (None, FAKE + 1)), (3, (None, FAKE + 2)),
                    (4, (FAKE + 2,)), (5, (None, FAKE + 64))):
        for bad in bads:
            a = list(m)
            a[i] = bad
            assert lib.kvq_evict_compact(ctypes.byref(c), ctypes.byref(p), *a, 1 << 40, None) == 1
    for other in (dict(num_blocks=9), dict(block_size=32, num_blocks=4), dict(num_kv_heads=1)):
        o = cache_desc(kvq, **other)
        assert lib.kvq_evict_compact(ctypes.byref(o), ctypes.byref(p), *m, 1 << 40, None) == 1


def test_masked_and_mass_refuse_token_counts_that_overflow(kvq):
    lib, c = kvq.load(), cache_desc(kvq)
    n = ctypes.c_size_t(0)
    for batch, tokens in ((0, 2 ** 31 - 1), (1, 2 ** 31 - 1), (1, 2 ** 30 + 1), (1024, 2 ** 20 + 1)):
        p = params(kvq, batch=batch, q_tokens=tokens)
        a = [ctypes.byref(c), ctypes.byref(p)]
        assert lib.kvq_attend_masked_workspace_size(*a, ctypes.byref(n)) == 2
        assert lib.kvq_key_mass_workspace_size(*a, ctypes.byref(n)) == 2


def test_evict_refuses_shapes_that_overflow(kvq):
    lib = kvq.load()
    for d in (dict(num_kv_heads=2 ** 14, block_size=2 ** 16), dict(batch=2 ** 20, num_kv_heads=32)):
        p = kvq.EvictParams(**{**dict(batch=2, max_blocks_per_seq=4, max_seq_len=0, num_blocks=8, block_size=16,
                                      num_kv_heads=2, budget=32, sinks=0, recent=0), **d})
        assert lib.kvq_evict_select(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE, FAKE + 4, None) == 2


def test_masked_refuses_an_output_over_the_queries(kvq):
    lib, c, p = kvq.load(), cache_desc(kvq), params(kvq)
    size = 2 * 5 * 8 * c.head_dim * 2
    for out in (FAKE, FAKE + 16, FAKE + size - 16, FAKE - size + 16):
        assert lib.kvq_attend_masked(ctypes.byref(c), ctypes.byref(p), None, FAKE, FAKE, FAKE, None, out, None, FAKE,
                                     1 << 40, None) == 1
