"""Masked attention and key mass at the edges of what their arguments allow,
against the 64-bit forms of score_ref.

The lse's bound (lse_bound): a logit takes at most 64 fp32 accumulations of
partial sums of at most `size` = sum |q k| sm_scale (2^6 * 2^-24), with a
per-channel K scale 2^-21 of it from the two f16 parts of the operand: together
2^-17.  A cap is below its argument and has a slope of at most 1: its own error
is 2^-21 of its value (tanh to 4e-7) and a rounding or two of its argument
(2^-23 of it), which the factor of 2 between 2^-17 and 2^-18 + 2^-21 leaves
room for.  The last roundings (bias, exp2, log2, the sum of the parts) are 2^-20
of 1, of the lse and of the largest bias that was taken out of it."""
import dataclasses

import numpy as np
import pytest
import torch

import score_ref as ref
from guard import guarded
from test_gpu_masked import CASES, check, dev, documents, gpu_cache, run, slopes_of

pytestmark = pytest.mark.gpu

INT8, FP8, INT4 = ref.INT8, ref.FP8, ref.INT4
TENSOR, CHANNEL = ref.TENSOR, ref.CHANNEL


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def lse_bound(c: ref.Cache, r_lse, size, slopes=None):
    far = 0.0 if slopes is None else max(abs(float(s)) for s in slopes) * max(c.case.lens)
    return 2.0 ** -17 * size + 2.0 ** -20 * (1 + np.abs(r_lse) + far)


def check_lse(c: ref.Cache, lse, slopes=None, key_begin=None, key_end=None):
    _, r_lse, _, _, size = ref.attend(c, slopes, key_begin, key_end)
    some = r_lse != -np.inf
    assert (lse[~some] == -np.inf).all() and np.isfinite(lse[some]).all()
    e = np.abs(lse[some] - r_lse[some]) / lse_bound(c, r_lse, size, slopes)[some]
    assert e.size == 0 or e.max() <= 1.0, f"lse {e.max():.2f} times its bound"


def mass_call(kvq, c: ref.Cache, lse, mass, decay=1.0, fresh=None, slopes=None, key_begin=None, key_end=None):
    case = c.case
    g = gpu_cache(kvq, c)
    B = len(case.lens)
    p = kvq.make_params(B, case.hq, case.c, c.width, softcap=case.softcap, window=case.window, sm_scale=case.sm_scale)
    ws = guarded(torch.zeros(kvq.kvq_key_mass_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda"), "ws")
    m = guarded(dev(mass), "mass")
    f32 = lambda a: None if a is None else dev(np.asarray(a, np.float32))  # noqa: E731
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    kvq.kvq_key_mass(g, p, kvq.ScoreMask(f32(slopes), i32(key_begin), i32(key_end)), dev(c.q).to(torch.bfloat16),
                     dev(c.table), dev(np.array(case.lens, np.int32)), dev(lse.astype(np.float32)), m, ws, decay=decay,
                     fresh=fresh)
    assert kvq.kvq_get_device_error() == 0
    return m.cpu().numpy()


# ------------------------------------------------------- ends of the intervals

@pytest.mark.parametrize("c,name", [(1, "int8 row d128"), (8, "fp8 row"), (90, "int8 row d256 g6"), (90, "fp8 row"),
                                    (90, "int4 channel d256"), (90, "int4 row"), (20, "fp8 tensor cap"),
                                    (3, "latent d576")])
@pytest.mark.parametrize("low", [-(2 ** 31), -(2 ** 31) + 100, -1])
def test_ends_far_below_zero(kvq, c, name, low):
    """Every second token's interval ends at or near the lowest int32 while the
    tokens beside it see keys: it sees nothing, on every layout."""
    case = dataclasses.replace(CASES[name], c=c, lens=(150, max(c, 97), max(c, 200)))
    cache = ref.Cache(case)
    pos = np.stack([L - c + np.arange(c) for L in case.lens])
    begin = np.zeros_like(pos)
    end = pos + 1
    begin[1, ::3] = low
    begin[2, ::5] = 2 ** 31 - 1
    for b in range(3):
        end[b, b % 2::2] = low
    s = slopes_of(case.hq)
    check(cache, run(kvq, cache, s, begin, end), s, begin, end)
    check(cache, run(kvq, cache, None, begin, end), None, begin, end)


@pytest.mark.parametrize("c,name", [(1, "int8 row d128"), (9, "fp8 row"), (40, "int8 row d256 g6"),
                                    (40, "int4 channel d256"), (5, "latent d576")])
def test_mass_of_ends_far_below_zero(kvq, c, name):
    case = dataclasses.replace(CASES[name], c=c, lens=(150, max(c, 97)))
    cache = ref.Cache(case)
    pos = np.stack([L - c + np.arange(c) for L in case.lens])
    end = pos + 1
    end[:, ::2] = -(2 ** 31)
    end[1, 1::4] = -(2 ** 31) + 65
    s = slopes_of(case.hq)
    lse = ref.attend(cache, s, None, end)[1]
    mass = np.random.default_rng(1).exponential(0.1, (cache.nb, case.hkv, case.bs)).astype(np.float32)
    got = mass_call(kvq, cache, lse, mass, 0.5, 0, s, None, end)
    want, tol = ref.key_mass(cache, lse.astype(np.float32), mass, 0.5, 0, s, None, end)
    assert (np.abs(got - want) <= tol).all()


# ---------------------------------------------------------------------- the cap

CAPPED = {
    "grouped d64": ref.Case(d=64, hq=4, hkv=4, lens=(130, 65), c=1),
    "grouped d128": ref.Case(dtype=FP8, lens=(333, 100), c=3),
    "grouped d256 group scales": ref.Case(dtype=INT4, km=ref.GROUP, vm=ref.GROUP, gs=32, d=256, lens=(150, 77), c=2),
    "wide d256": ref.Case(d=256, hq=16, hkv=2, lens=(257, 64), c=4),
    "wide channel d256": ref.Case(dtype=INT4, km=CHANNEL, vm=CHANNEL, d=256, hq=12, hkv=2, lens=(190, 64), c=4),
    "wide d576": ref.Case(d=576, hq=8, hkv=1, latent=True, dv=512, lens=(99, 140), c=2),
    "tile d128": ref.Case(dtype=FP8, lens=(333, 100), c=40),
    "tile tensor d128": ref.Case(dtype=INT8, km=TENSOR, vm=TENSOR, lens=(130, 97), c=33),
    "tile channel d128": ref.Case(km=CHANNEL, vm=CHANNEL, lens=(333, 100), c=40),
    "tile channel d256": ref.Case(dtype=INT4, km=CHANNEL, vm=CHANNEL, d=256, hq=14, hkv=2, lens=(190, 70), c=50),
    "tile d256": ref.Case(d=256, hq=6, hkv=1, lens=(190, 70), c=50),
}


@pytest.mark.parametrize("cap", [5.0, 500.0, 20000.0])
@pytest.mark.parametrize("name", CAPPED)
def test_lse_under_a_cap(kvq, name, cap):
    """The lse is fp32-accurate under a cap of any size: the cap's own error is
    relative to the capped logit, not to the cap.  Under a steep bias, where few
    keys carry a row and their errors do not average out, and without one."""
    cache = ref.Cache(dataclasses.replace(CAPPED[name], softcap=cap))
    for s in ([0.5] * cache.case.hq, None):
        got = run(kvq, cache, s)
        check_lse(cache, got[1], s)
        check(cache, got, s)


@pytest.mark.parametrize("cap", [5.0, 500.0, 20000.0])
@pytest.mark.parametrize("name", CAPPED)
def test_attention_and_mass_cap_alike(kvq, name, cap):
    """The weights that the attention's own lse gives a row's keys add up to 1:
    the two calls give a key the same score."""
    cache = ref.Cache(dataclasses.replace(CAPPED[name], softcap=cap))
    case = cache.case
    s = [0.5] * case.hq
    lse = run(kvq, cache, s)[1]
    got = mass_call(kvq, cache, lse, np.zeros((cache.nb, case.hkv, case.bs), np.float32), slopes=s)
    _, r_lse, _, _, size = ref.attend(cache, s)
    # each weight moves by what its logit and the lse are off (their bound, twice),
    # and by 2^-20 for exp2 and the sums
    bound = 2 * lse_bound(cache, r_lse, size, s) + 2.0 ** -20
    for b in range(len(case.lens)):
        blk, row = cache.rows(b)
        for h in range(case.hkv):
            heads = slice(h * case.group, (h + 1) * case.group)
            assert abs(got[blk, h, row].astype(np.float64).sum() - case.c * case.group) <= bound[b, :, heads].sum()


# ------------------------------------------------------------ ends of the range

RANGE = {
    "int8 d128": ref.Case(lens=(333, 100)),
    "fp8 d256": ref.Case(dtype=FP8, d=256, hq=12, hkv=2, lens=(333, 90)),
    "int4 d256": ref.Case(dtype=INT4, d=256, hq=8, hkv=2, lens=(200, 90)),
}


def far_cache(case, p):
    """K rows of about 2^p and queries of about 2^-p: ordinary logits."""
    cache = ref.Cache(case)
    cache.k_scale *= np.float32(2.0 ** p)
    cache.q = ref.bf16(cache.q * np.float32(2.0 ** -p))
    return cache


@pytest.mark.parametrize("p", [100, 122])
@pytest.mark.parametrize("c", [1, 40])
@pytest.mark.parametrize("name", RANGE)
def test_large_keys_and_small_queries(kvq, name, c, p):
    """The logit factor of a row may be small and the K scale large: neither is
    cut off, and no product of the two leaves fp32's range on the way."""
    cache = far_cache(dataclasses.replace(RANGE[name], c=c), p)
    s = slopes_of(cache.case.hq)
    got = run(kvq, cache, s)
    check_lse(cache, got[1], s)
    check(cache, got, s)


@pytest.mark.parametrize("c,call", [(8, "decode"), (2, "decode"), (40, "prefill")])
@pytest.mark.parametrize("name", RANGE)
def test_large_keys_and_small_queries_without_a_rule(kvq, name, c, call):
    cache = far_cache(dataclasses.replace(RANGE[name], c=c), 100)
    case = cache.case
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(2, case.hq, c, cache.width)
    q, table, lens = dev(cache.q).to(torch.bfloat16), dev(cache.table), dev(np.array(case.lens, np.int32))
    out = torch.zeros((2, c, case.hq, case.d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, c, case.hq), device="cuda")
    if call == "decode":
        out, lse = kvq.decode_step(g, p, q, table, lens, kvq.alloc_decode_buffers(g, p))
    else:
        ws = torch.zeros(kvq.kvq_prefill_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
        kvq.kvq_prefill(g, p, q, table, lens, None, out, lse, ws)
    assert kvq.kvq_get_device_error() == 0
    r_lse, size = ref.attend(cache)[1], ref.attend(cache)[4]
    # (the tensor-memory decode sums its weights as f16, each 2^-11 off: the sum,
    # and so the lse, by 2^-11 at most)
    assert (np.abs(lse.double().cpu().numpy() - r_lse) <= lse_bound(cache, r_lse, size) + 2.0 ** -11).all()
    check(cache, (out.double().cpu().numpy(), r_lse))


@pytest.mark.parametrize("p", [100, 122])
@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("c", [1, 40])
@pytest.mark.parametrize("name", RANGE)
def test_mass_of_large_keys_and_small_queries(kvq, name, c, cap, p):
    """A padding token among the rows, whose logit factor is 0."""
    cache = far_cache(dataclasses.replace(RANGE[name], c=c, softcap=cap), p)
    case = cache.case
    end = np.stack([L - c + np.arange(c) + 1 for L in case.lens])
    if c > 1:
        end[:, 3] = 0
    lse = ref.attend(cache, None, None, end)[1]
    got = mass_call(kvq, cache, lse, np.zeros((cache.nb, case.hkv, case.bs), np.float32), key_end=end)
    want, tol = ref.key_mass(cache, lse.astype(np.float32), np.zeros_like(got), 1.0, case.c, None, None, end)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()


# --------------------------------------------------- lse of a per-channel scale

@pytest.mark.parametrize("dtype", [INT8, FP8, INT4])
@pytest.mark.parametrize("d,c,hq,hkv", [(64, 5, 7, 1), (128, 1, 10, 2), (128, 40, 7, 1), (128, 40, 9, 3),
                                        (256, 5, 10, 2), (256, 20, 7, 1), (256, 40, 20, 4), (256, 70, 3, 1),
                                        (576, 3, 7, 1)])
@pytest.mark.parametrize("sign", [0.5, -0.5])
def test_lse_of_a_per_channel_scale_under_a_rule(kvq, dtype, d, c, hq, hkv, sign):
    """The two-part operand with odd groups, documents, prefixes, biases of both
    signs and a sink: an f16 operand of one part would be 2^-11 of sum |q k| off."""
    if d == 576 and dtype == INT4:
        pytest.skip("576-channel rows are 8-bit")
    case = ref.Case(dtype=dtype, km=CHANNEL, vm=CHANNEL, d=d, c=c, hq=hq, hkv=hkv, lens=(160, max(c, 64)),
                    latent=d == 576, dv=512 if d == 576 else 0)
    cache = ref.Cache(case)
    begin, end = documents(case, (13, 40, 64, 90))
    end[1] = np.maximum(end[1], 30)  # a prefix, seen in both directions
    begin[1] = np.minimum(begin[1], 8)
    end[0, ::7] = 0
    s = [sign] * hq
    sink = np.linspace(-2.0, 2.0, hq)
    got = run(kvq, cache, s, begin, end, sink)
    check_lse(cache, got[1], s, begin, end)
    check(cache, got, s, begin, end, sink)


# -------------------------------------------------------------------- head sinks

@pytest.mark.parametrize("name", ["int8 row d128", "fp8 tensor cap", "int4 channel d256"])
@pytest.mark.parametrize("c", [1, 40])
def test_mass_beside_a_sink(kvq, name, c):
    """With a head sink the attention's weights are e^(s - log(e^lse + e^sink)):
    kvq_key_mass takes that logarithm in the lse's place."""
    case = dataclasses.replace(CASES[name], c=c, lens=(130, max(c, 64)))
    cache = ref.Cache(case)
    sink = np.linspace(-1.0, 3.0, case.hq)
    lse = ref.attend(cache)[1]
    both = np.logaddexp(lse, sink)
    zero = np.zeros((cache.nb, case.hkv, case.bs), np.float32)
    got = mass_call(kvq, cache, both, zero)
    want, tol = ref.key_mass(cache, both.astype(np.float32), zero, 1.0, c)
    assert (np.abs(got - want) <= tol).all()
    for b, L in enumerate(case.lens):
        blk, row = cache.rows(b)
        total = got[blk, :, row].astype(np.float64).sum()
        share = (1.0 / (1.0 + np.exp(sink - lse[b]))).sum()  # what the sink leaves of each row
        assert abs(total - share) <= tol[blk, :, row].sum() + 2.0 ** -22 * case.c * case.hq * (1 + np.abs(both).max())


# ------------------------------------------------------------- freed pages

@pytest.mark.parametrize("name,c", [("int8 row d128", 1), ("fp8 row", 5), ("int8 row d256 g6", 40), ("fp8 row", 40),
                                    ("int4 channel d256", 40), ("latent d576", 3), ("int8 channel d64", 6)])
@pytest.mark.parametrize("how", ["window", "documents"])
def test_pages_before_every_key_that_is_seen(kvq, name, c, how):
    """Pages whose rows lie wholly before the first key that a token sees, down to
    the last one, may have left the table: they are neither read nor flagged."""
    case = dataclasses.replace(CASES[name], c=c, bs=16, lens=(250, 241), window=30 if how == "window" else 0)
    cache = ref.Cache(case)
    begin = None
    if how == "documents":
        begin = np.array([[L - c - 30] * c for L in case.lens], np.int32)
    want = ref.attend(cache, None, begin)
    for b, L in enumerate(case.lens):
        first = L - c + 1 - 30 if how == "window" else L - c - 30
        cache.table[b, :first // 16] = -1
    g = gpu_cache(kvq, cache)
    got = run(kvq, cache, None, begin, gcache=g)
    assert (np.abs(got[1] - want[1]) <= lse_bound(cache, want[1], want[4]) + 2.0 ** -15).all()
    tol = 2.0 ** -8 * np.abs(want[0]) + want[3] + 2 * (2.0 ** -11 * want[4] + 2.0 ** -15)[..., None] * want[2] + 1e-30
    assert (np.abs(got[0] - want[0]) <= tol).all()


# ------------------------------------------------------------------ steep biases

@pytest.mark.parametrize("slope", [0.25, 30.0, 1000.0])
@pytest.mark.parametrize("d,km,c,hq,hkv,cap", [(128, ref.ROW, 1, 8, 2, 0.0), (128, ref.ROW, 70, 8, 2, 0.0),
                                               (256, CHANNEL, 70, 6, 1, 0.0), (256, ref.ROW, 70, 6, 1, 30.0),
                                               (64, ref.ROW, 5, 4, 1, 0.0), (256, ref.ROW, 4, 16, 2, 0.0)])
def test_steep_biases(kvq, slope, d, km, c, hq, hkv, cap):
    """A bias is slope times distance to a rounding or two of itself; in the tile
    kernel to 2^-14 of the slope.  (Some tokens sit on the last key of a tile,
    some see no key near.)"""
    case = ref.Case(d=d, km=km, vm=km, c=c, hq=hq, hkv=hkv, lens=(192, 230), softcap=cap)
    cache = ref.Cache(case)
    pos = np.stack([L - c + np.arange(c) for L in case.lens])
    end = pos + 1
    end[:, ::3] -= 5
    s = [slope] * hq
    lse = run(kvq, cache, s, None, end)[1]
    _, r_lse, _, _, size = ref.attend(cache, s, None, end)
    # (slope times an integer below 2^24 is rounded once where the anchor's bias
    # goes back into the lse; that is in 2^-20 of the lse.  The tile kernel takes
    # up to 63 slopes a tile from a rounded base in at most 8 rounded steps: 9
    # times half an ulp, 2^-24 of 64 slopes, is below 2^-14 of the slope)
    tile = d >= 128 and c * (hq // hkv) > 16
    bound = 2.0 ** -17 * size + 2.0 ** -20 * (1 + np.abs(r_lse)) + (2.0 ** -14 * slope if tile else 0.0)
    assert (np.abs(lse - r_lse) <= bound).all()


# ------------------------------------------------------------ mixed scale modes

@pytest.mark.parametrize("km,vm", [(CHANNEL, ref.GROUP), (ref.GROUP, CHANNEL), (ref.ROW, ref.GROUP), (CHANNEL, ref.ROW)])
@pytest.mark.parametrize("d,c,hq,hkv", [(128, 1, 8, 2), (128, 9, 7, 1), (256, 20, 6, 3), (64, 3, 4, 4)])
def test_scale_modes_of_two_kinds(kvq, km, vm, d, c, hq, hkv):
    """K and V of different modes, with and without the two-part operand."""
    case = ref.Case(dtype=INT4, km=km, vm=vm, gs=32, d=d, c=c, hq=hq, hkv=hkv, lens=(140, max(c, 33)))
    cache = ref.Cache(case)
    begin, end = documents(case, (13, 40, 90))
    s = slopes_of(hq, -1.0)
    got = run(kvq, cache, s, begin, end)
    check_lse(cache, got[1], s, begin, end)
    check(cache, got, s, begin, end)


# ------------------------------------------------------------------- repetition

@pytest.mark.parametrize("name,c", [("int8 row d128", 1), ("fp8 tensor cap", 8), ("fp8 row", 40),
                                    ("int4 channel d256", 40), ("int8 row d256 g6", 90), ("latent d576", 3)])
def test_repeated_calls_give_the_same_bits(kvq, name, c):
    case = dataclasses.replace(CASES[name], c=c, lens=(1500, 700, max(c, 97)))
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    s = slopes_of(case.hq)
    begin, end = documents(case, (13, 400, 900))
    first = run(kvq, cache, s, begin, end, gcache=g)
    for _ in range(4):
        again = run(kvq, cache, s, begin, end, gcache=g)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
