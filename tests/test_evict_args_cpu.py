"""The eviction calls refuse outputs that overlap one another or an input, on the
host and before any launch: the CTAs of a head each read its length, a selection
reads its weights more than once, and the threads that move a unit of rows each
read where it lies."""
import ctypes

import pytest

FAKE = 0x7F0000000000  # addresses that are never dereferenced on the host
B, HKV, BS, WIDTH, NB, BUDGET = 3, 2, 16, 8, 64, 20
SIZES = {"mass": 4 * NB * HKV * BS, "block_table": 4 * B * WIDTH, "seq_lens": 4 * B, "keep": 4 * B * HKV * BUDGET,
         "kept_lens": 4 * B}
ORDER = ("mass", "block_table", "seq_lens", "keep", "kept_lens")


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import build, kvq
    build.build()
    kvq.load()
    return kvq


def select(kvq, at):
    p = kvq.make_evict_params(B, WIDTH, BUDGET, num_blocks=NB, block_size=BS, num_kv_heads=HKV)
    return kvq.load().kvq_evict_select(ctypes.byref(p), *(at[n] for n in ORDER), None)


@pytest.mark.parametrize("out,other", [("kept_lens", "seq_lens"), ("kept_lens", "block_table"), ("kept_lens", "mass"),
                                       ("kept_lens", "keep"), ("keep", "seq_lens"), ("keep", "block_table"),
                                       ("keep", "mass")])
def test_overlapping_outputs_are_refused(kvq, out, other):
    at = {n: FAKE + (i << 20) for i, n in enumerate(ORDER)}
    # the same address; the first and the last element shared; one inside the other
    for a in {at[other], at[other] + SIZES[other] - 4, at[other] - SIZES[out] + 4, at[other] + 4}:
        assert select(kvq, {**at, out: a}) == 1


COMPACT = {"k_codes": NB * HKV * BS * 64, "v_codes": NB * HKV * BS * 64, "k_scale": 4 * NB * HKV * BS,
           "v_scale": 4 * NB * HKV * BS, "block_table": 4 * B * WIDTH, "dst_table": 4 * B * WIDTH,
           "keep": 4 * B * HKV * BUDGET, "kept_lens": 4 * B, "mass": 4 * NB * HKV * BS, "workspace": 4096}


@pytest.mark.parametrize("read", ["block_table", "dst_table", "keep", "kept_lens"])
@pytest.mark.parametrize("written", ["k_codes", "v_codes", "k_scale", "v_scale", "mass"])
def test_moving_rows_over_their_own_places_is_refused(kvq, read, written):
    p = kvq.make_evict_params(B, WIDTH, BUDGET, num_blocks=NB, block_size=BS, num_kv_heads=HKV)
    base = {n: FAKE + (i << 20) for i, n in enumerate(COMPACT)}
    for a in {base[written], base[written] + COMPACT[written] - 4, base[written] - COMPACT[read] + 4}:
        at = {**base, read: a}
        c = kvq.CacheDesc(kvq.INT8, kvq.PER_ROW, kvq.PER_ROW, NB, BS, HKV, 64, at["k_codes"], at["v_codes"],
                          at["k_scale"], at["v_scale"])
        st = kvq.load().kvq_evict_compact(ctypes.byref(c), ctypes.byref(p), at["block_table"], at["dst_table"],
                                          at["keep"], at["kept_lens"], at["mass"], at["workspace"],
                                          COMPACT["workspace"], None)
        assert st == 1
