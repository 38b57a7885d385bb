"""Attention under a score rule (kvq_attend_masked) against its 64-bit form:
distance biases, document / prefix / padding intervals, odd chunk lengths,
every cache type and scale mode, rows that see nothing, and cache rows that no
token sees holding NaN.

Tolerances, per output channel: bf16 rounding of the result is at most 2^-8 of
it (half of finfo(bf16).eps); the weights and, with per-row V scales, the
scaled values or weights are rounded to f16 (2^-11 each) of a mean absolute
value A = sum p |v|, and those below 2^-14 to 2^-25 each (score_ref.attend
adds these up); a logit is off by at most 2^-11 of sum |q k| when a
per-channel K scale is folded into an f16 query, else by 2^-15 (the cap's
tanh, 50 x a few 1e-7, and fp32 sums), which moves o by at most 2 A times it."""
import numpy as np
import pytest
import torch

import score_ref as ref
from guard import guarded

pytestmark = pytest.mark.gpu

INT8, FP8, INT4 = ref.INT8, ref.FP8, ref.INT4
ROW, TENSOR, CHANNEL, GROUP = ref.ROW, ref.TENSOR, ref.CHANNEL, ref.GROUP


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def gpu_cache(kvq, c: ref.Cache):
    case = c.case
    static = lambda m, s: dev(s) if m in (TENSOR, CHANNEL) else None  # noqa: E731
    g = kvq.QuantizedPagedCache(case.dtype, case.km, case.vm, c.nb, case.bs, case.hkv, case.d,
                                k_static=static(case.km, c.k_scale), v_static=static(case.vm, c.v_scale),
                                latent=case.latent, v_head_size=case.dv, group_size=case.gs)
    g.k_codes.copy_(dev(c.k_codes))
    g.k_scale.copy_(dev(c.k_scale).reshape(g.k_scale.shape))
    if not case.latent:
        g.v_codes.copy_(dev(c.v_codes))
        g.v_scale.copy_(dev(c.v_scale).reshape(g.v_scale.shape))
    return g


def run(kvq, c: ref.Cache, slopes=None, key_begin=None, key_end=None, sink=None, flags=0, gcache=None):
    case = c.case
    g = gcache or gpu_cache(kvq, c)
    B = len(case.lens)
    p = kvq.make_params(B, case.hq, case.c, c.width, softcap=case.softcap, window=case.window,
                        sm_scale=case.sm_scale, flags=flags)
    n = kvq.kvq_attend_masked_workspace_size(g, p)
    ws = guarded(torch.zeros(n // 4, dtype=torch.int32, device="cuda"), "workspace")
    out = guarded(torch.full((B, case.c, case.hq, g.out_dim), 7.0, dtype=torch.bfloat16, device="cuda"), "out")
    lse = guarded(torch.full((B, case.c, case.hq), 7.0, device="cuda"), "lse")
    f32 = lambda a: None if a is None else dev(np.asarray(a, np.float32))  # noqa: E731
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    mask = None
    if slopes is not None or key_begin is not None or key_end is not None:
        mask = kvq.ScoreMask(f32(slopes), i32(key_begin), i32(key_end))
    kvq.kvq_attend_masked(g, p, mask, dev(c.q).to(torch.bfloat16), dev(c.table), dev(np.array(case.lens, np.int32)),
                          f32(sink), out, lse, ws)
    assert kvq.kvq_get_device_error() == 0
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def check(c: ref.Cache, got, slopes=None, key_begin=None, key_end=None, sink=None):
    out, lse = got
    r_out, r_lse, absv, f16, size = ref.attend(c, slopes, key_begin, key_end, sink)
    ds = (2.0 ** -11 * size if c.case.km == CHANNEL else np.zeros_like(size)) + 2.0 ** -15
    empty = r_lse == -np.inf
    assert (lse[empty] == -np.inf).all() and np.isfinite(lse[~empty]).all()
    assert (out[empty] == 0).all() and np.isfinite(out).all()
    e = np.abs(lse[~empty] - r_lse[~empty]) - (ds[~empty] + 2.0 ** -20 * (1 + np.abs(r_lse[~empty])))
    assert e.size == 0 or e.max() <= 0, f"lse off by {e.max():.2e} more than its bound"
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    worst = (np.abs(out - r_out) / tol).max()
    assert worst <= 1.0, f"output {worst:.2f} times its bound"


def slopes_of(hq, sign=1.0):
    return [sign * 2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]


def documents(case, cuts):
    """key_begin / key_end of documents that begin at `cuts` of every sequence."""
    begin = np.zeros((len(case.lens), case.c), np.int32)
    end = np.zeros_like(begin)
    for b, L in enumerate(case.lens):
        for t in range(case.c):
            pos = L - case.c + t
            begin[b, t] = max([0] + [x for x in cuts if x <= pos])
            end[b, t] = pos + 1
    return begin, end


# decode-sized and prompt-sized chunks on every kernel layout: (case, what)
CASES = {
    "int8 row d128": ref.Case(lens=(100, 1, 333)),
    "int8 row d256 g6": ref.Case(d=256, hq=12, lens=(257, 64), bs=32),
    "int8 channel d64": ref.Case(d=64, km=CHANNEL, vm=TENSOR, lens=(70, 65), hq=4, hkv=4),
    "fp8 tensor cap": ref.Case(dtype=FP8, km=TENSOR, vm=TENSOR, lens=(130, 31), softcap=50.0),
    "fp8 row": ref.Case(dtype=FP8, lens=(129, 200)),
    "int4 channel d256": ref.Case(dtype=INT4, km=CHANNEL, vm=CHANNEL, d=256, lens=(190,), hq=6, hkv=1),
    "int4 row": ref.Case(dtype=INT4, lens=(95, 64), d=64),
    "int4 group": ref.Case(dtype=INT4, km=GROUP, vm=GROUP, gs=32, lens=(150, 77)),
    "int8 group k, row v": ref.Case(km=GROUP, vm=ROW, gs=64, d=256, lens=(150, 17)),
    "fp8 group v": ref.Case(dtype=FP8, km=TENSOR, vm=GROUP, gs=128, lens=(150, 17)),
    "latent d256": ref.Case(d=256, hq=8, hkv=1, latent=True, dv=192, lens=(99, 140)),
    "latent d576": ref.Case(d=576, hq=8, hkv=1, latent=True, dv=512, lens=(99, 140)),
    "latent d576 fp8": ref.Case(dtype=FP8, km=TENSOR, vm=TENSOR, d=576, hq=6, hkv=1, latent=True, dv=512, lens=(130,)),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("c", [1, 3, 8, 19, 70])
def test_bias_and_documents(kvq, name, c):
    import dataclasses
    base = CASES[name]
    case = dataclasses.replace(base, c=c, seed=c, lens=tuple(max(L, c) if c > 8 else L for L in base.lens))
    cache = ref.Cache(case)
    s = slopes_of(case.hq)
    begin, end = documents(case, (13, 40, 64, 90))
    check(cache, run(kvq, cache, slopes=s, key_begin=begin, key_end=end), s, begin, end)


@pytest.mark.parametrize("name", ["int8 row d128", "int8 row d256 g6", "fp8 tensor cap", "int4 channel d256",
                                  "latent d576", "int8 channel d64"])
@pytest.mark.parametrize("c", [1, 7, 65, 130])
def test_prefix_and_sink(kvq, name, c):
    """The prefix is seen in both directions; the last tokens' window still
    ends where the prefix does."""
    import dataclasses
    base = CASES[name]
    case = dataclasses.replace(base, c=c, seed=3 * c, lens=tuple(max(L, c + 5) for L in base.lens))
    cache = ref.Cache(case)
    B = len(case.lens)
    end = np.stack([np.maximum(L - c + np.arange(c) + 1, L // 2) for L in case.lens]).astype(np.int32)
    sink = np.linspace(-1, 2, case.hq)
    s = slopes_of(case.hq)
    s[0] = 0.0
    check(cache, run(kvq, cache, slopes=s, key_end=end, sink=sink), s, None, end, sink)
    assert B == end.shape[0]


@pytest.mark.parametrize("c", [1, 5, 40])
@pytest.mark.parametrize("name", ["int8 row d128", "fp8 row", "latent d576"])
def test_no_rule_is_causal_attention(kvq, name, c):
    """mask NULL equals an empty ScoreMask, and both the causal rule with the window."""
    import dataclasses
    case = dataclasses.replace(CASES[name], c=c, window=37, lens=(120, 41))
    cache = ref.Cache(case)
    a = run(kvq, cache)
    check(cache, a)
    end = np.stack([L - c + np.arange(c) + 1 for L in case.lens])
    b = run(kvq, cache, key_end=end)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("c,name", [(1, "int8 row d128"), (6, "fp8 row"), (90, "int8 row d256 g6"), (90, "fp8 row"),
                                    (3, "latent d576"), (8, "int8 group k, row v"), (90, "int4 row")])
def test_rows_that_see_nothing(kvq, c, name):
    """Empty intervals, reversed ones, ones outside the sequence, in the middle
    of a group and for whole groups and sequences."""
    import dataclasses
    case = dataclasses.replace(CASES[name], c=c, lens=(150, max(c, 97), max(c, 20)))
    cache = ref.Cache(case)
    r = np.random.default_rng(5)
    begin = r.integers(-5, 60, (3, c)).astype(np.int32)
    end = r.integers(-9, 200, (3, c)).astype(np.int32)
    end[0, ::3] = begin[0, ::3]
    begin[1] = 2 ** 31 - 1
    end[2] = -(2 ** 31)
    begin[0, -1], end[0, -1] = -(2 ** 31), 2 ** 31 - 1
    s = slopes_of(case.hq)
    check(cache, run(kvq, cache, s, begin, end), s, begin, end)


@pytest.mark.parametrize("c", [1, 8, 66])
def test_far_keys_keep_their_weights(kvq, c):
    """Every visible key lies far behind the query under a steep bias: the
    biases are around -2^13 and the weights still resolve, as they would
    next to the query.  Negative slopes favour the furthest key."""
    case = ref.Case(lens=(9000,), c=c, bs=256, d=128)
    cache = ref.Cache(case)
    begin = np.full((1, c), 40, np.int32)
    end = np.full((1, c), 171, np.int32)
    for sign in (1.0, -1.0):
        s = [sign * x for x in (1.0, 0.7, 0.5, 0.3, 0.2, 0.1, 0.05, 1.5)]
        out, lse = run(kvq, cache, s, begin, end)
        r_out, r_lse, absv, f16, _ = ref.attend(cache, s, begin, end)
        # lse itself is fp32 around -1.3e4: 2^-24 of it, and of slope * distance
        assert np.abs(lse - r_lse).max() <= 2.0 ** -22 * np.abs(r_lse).max() + 2.0 ** -15
        tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2.0 ** -14 * absv
        assert (np.abs(out - r_out) <= tol).all()


@pytest.mark.parametrize("c", [1, 4, 20, 100])
@pytest.mark.parametrize("name", ["int8 row d128", "fp8 row", "int4 group", "int8 row d256 g6", "latent d576"])
def test_junk_in_rows_that_no_token_sees(kvq, name, c):
    """Left padding below every interval and a gap between two documents hold
    NaN and huge scales and NaN codes: nothing of them reaches an output."""
    import dataclasses
    case = dataclasses.replace(CASES[name], c=c, lens=(260,), seed=11)
    cache = ref.Cache(case)
    begin = np.zeros((1, c), np.int32)
    end = np.zeros((1, c), np.int32)
    for t in range(c):
        pos = 260 - c + t
        begin[0, t], end[0, t] = (37, 100) if t % 2 else (181, pos + 1)
    if c == 1:
        begin[0, 0], end[0, 0] = 37, 100
    seen = np.zeros(260, bool)
    for t in range(c):
        seen[begin[0, t]:end[0, t]] = True
    s = slopes_of(case.hq)
    expect = ref.attend(cache, s, begin, end)
    blk, row = cache.rows(0)
    for side in ("k", "v"):
        codes, scale = getattr(cache, side + "_codes"), getattr(cache, side + "_scale")
        bad = np.flatnonzero(~seen)
        if case.dtype == FP8:
            codes[blk[bad], :, row[bad]] = 0x7F
        if scale.ndim >= 3:
            scale[blk[bad[0::3]], :, row[bad[0::3]]] = np.nan
            scale[blk[bad[1::3]], :, row[bad[1::3]]] = np.inf
            scale[blk[bad[2::3]], :, row[bad[2::3]]] = 1e38
    got = run(kvq, cache, s, begin, end)
    r_out, r_lse, absv, f16, size = expect
    assert np.isfinite(got[0]).all()
    ds = (2.0 ** -11 * size if case.km == CHANNEL else np.zeros_like(size)) + 2.0 ** -15
    tol = 2.0 ** -8 * np.abs(r_out) + f16 + 2 * ds[..., None] * absv + 1e-30
    assert (np.abs(got[0] - r_out) <= tol).all()


def test_many_groups_take_several_launches(kvq):
    """A chunk of more groups than one launch holds (8 tokens a group at
    head_dim 64): 8200 tokens, checked at the launches' seams."""
    case = ref.Case(d=64, hq=1, hkv=1, lens=(8300,), c=8200, bs=64)
    cache = ref.Cache(case)
    begin = np.maximum(0, np.arange(100, 8300) - 50).astype(np.int32)[None]
    out, lse = run(kvq, cache, [0.25], begin)
    pick = [0, 1, 7, 8, 4095, 8183, 8191, 8192, 8193, 8199]
    small = ref.Case(d=64, hq=1, hkv=1, lens=(8300,), c=8200, bs=64)
    for t in pick:
        lo, hi, pos = ref.visible(small, 0, t, begin, None)
        k, v = cache.values(0, 0, "k")[lo:hi], cache.values(0, 0, "v")[lo:hi]
        s = k @ cache.q[0, t, 0].astype(float) * case.scale - 0.25 * np.abs(pos - np.arange(lo, hi))
        p = np.exp(s - s.max())
        assert abs(lse[0, t, 0] - (s.max() + np.log(p.sum()))) <= 2.0 ** -14
        p /= p.sum()
        f16 = 2.0 ** -10 * (p @ np.abs(v)) + 2.0 ** -24 * (hi - lo) * cache.largest(0, 0, lo, hi)
        tol = 2.0 ** -8 * np.abs(p @ v) + f16 + 2.0 ** -14 * (p @ np.abs(v))
        assert (np.abs(out[0, t, 0] - p @ v) <= tol).all()


def test_short_sequences_and_batch_zero(kvq):
    """Sequences shorter than the chunk and empty ones; a batch of none."""
    case = ref.Case(lens=(0, 3, 40), c=12)
    cache = ref.Cache(case)
    check(cache, run(kvq, cache, slopes_of(8)), slopes_of(8))
    case = ref.Case(lens=(0, 30, 200), c=100, d=256)
    cache = ref.Cache(case)
    check(cache, run(kvq, cache, slopes_of(8)), slopes_of(8))
    p = kvq.make_params(0, 8, 5, 4)
    g = gpu_cache(kvq, cache)
    e = torch.empty((0, 5, 8, 256), dtype=torch.bfloat16, device="cuda")
    kvq.kvq_attend_masked(g, p, None, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                          torch.empty((0,), dtype=torch.int32, device="cuda"), None, e, None,
                          torch.empty(256, dtype=torch.int32, device="cuda"))


def test_bad_lengths_and_block_ids_are_flagged(kvq):
    case = ref.Case(lens=(50, 60), c=3)
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(2, 8, 3, cache.width)
    ws = torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 3, 8, 128), dtype=torch.bfloat16, device="cuda")
    q = dev(cache.q).to(torch.bfloat16)
    args = (out, None, ws)
    kvq.kvq_attend_masked(g, p, None, q, dev(cache.table), dev(np.array([50, -1], np.int32)), None, *args)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SEQ_LEN
    kvq.kvq_attend_masked(g, p, None, q, dev(cache.table), dev(np.array([10 ** 6, 60], np.int32)), None, *args)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SEQ_LEN
    bad = cache.table.copy()
    bad[0, 1], bad[1, 0] = -7, cache.nb
    kvq.kvq_attend_masked(g, p, None, q, dev(bad), dev(np.array([50, 60], np.int32)), None, *args)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_ID


@pytest.mark.parametrize("c", [1, 70])
def test_captured_and_on_another_stream(kvq, c):
    """Replays of a captured call, and a call on a side stream, give the bits of
    the plain call; two replayed graphs with workspaces of their own may overlap."""
    case = ref.Case(lens=(300, 211), c=c, d=128)
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(2, 8, c, cache.width)
    s = dev(np.array(slopes_of(8), np.float32))
    q, table = dev(cache.q).to(torch.bfloat16), dev(cache.table)
    lens = dev(np.array(case.lens, np.int32))
    n = kvq.kvq_attend_masked_workspace_size(g, p) // 4

    def bufs():
        return (torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros((2, c, 8), device="cuda"),
                torch.zeros(n, dtype=torch.int32, device="cuda"))

    def call(out, lse, ws, stream=None):
        kvq.kvq_attend_masked(g, p, kvq.ScoreMask(slopes=s), q, table, lens, None, out, lse, ws, stream)

    plain = bufs()
    call(*plain)
    side = bufs()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(*side, stream=st)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        b = bufs()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(*b)
        graphs.append(gr)
        outs.append(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_error() == 0
    for b in (side, *outs):
        assert torch.equal(plain[0], b[0]) and torch.equal(plain[1], b[1])


def test_refuses_wrong_tensors(kvq):
    case = ref.Case(lens=(50,), c=2)
    cache = ref.Cache(case)
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(1, 8, 2, cache.width)
    ws = torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    q, table = dev(cache.q).to(torch.bfloat16), dev(cache.table)
    lens, out = dev(np.array([50], np.int32)), torch.zeros((1, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    bad = [
        dict(q=q.float()), dict(q=q[:, :1]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
        dict(table=table.long()), dict(lens=lens.cpu()), dict(out=out.float()),
        dict(mask=kvq.ScoreMask(slopes=torch.zeros(7, device="cuda"))),
        dict(mask=kvq.ScoreMask(key_begin=torch.zeros((1, 3), dtype=torch.int32, device="cuda"))),
        dict(mask=kvq.ScoreMask(key_end=torch.zeros((1, 2), dtype=torch.int64, device="cuda"))),
        dict(lse=torch.zeros((1, 2, 9), device="cuda")), dict(ws=ws.cpu()),
    ]
    for kw in bad:
        a = dict(mask=None, q=q, table=table, lens=lens, out=out, lse=None, ws=ws)
        a.update(kw)
        with pytest.raises(ValueError):
            kvq.kvq_attend_masked(g, p, a["mask"], a["q"], a["table"], a["lens"], None, a["out"], a["lse"], a["ws"])
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_attend_masked(g, p, None, q, table, lens, None, out, None, ws[:16])
    assert e.value.status == 3


def test_many_tiles_take_several_launches(kvq):
    """More tiles of 128 rows than one launch holds: 16,500 tokens of 8 heads,
    checked at the launches' seam, in split and in whole units."""
    C, L = 16500, 16700
    case = ref.Case(d=128, hq=8, hkv=1, lens=(L,), c=C, bs=256)
    cache = ref.Cache(case)
    pos = np.arange(L - C, L)
    begin = np.maximum(0, pos - 300).astype(np.int32)[None]
    begin[0, 5000:5100] = 0
    s = slopes_of(8)
    sink = np.linspace(-1, 1, 8)
    out, lse = run(kvq, cache, s, begin, sink=sink)
    for t in (0, 1, 4999, 5050, 16383, 16384, 16385, 16399, 16400, 16499):
        lo, hi, p = ref.visible(case, 0, t, begin, None)
        k, v = cache.values(0, 0, "k")[lo:hi], cache.values(0, 0, "v")[lo:hi]
        f16c = 2.0 ** -24 * (hi - lo) * cache.largest(0, 0, lo, hi)
        for h in range(8):
            x = k @ cache.q[0, t, h].astype(float) * case.scale - s[h] * np.abs(p - np.arange(lo, hi))
            w = np.exp(x - x.max())
            l = x.max() + np.log(w.sum())
            assert abs(lse[0, t, h] - l) <= 2.0 ** -14
            w = w / w.sum() / (1 + np.exp(sink[h] - l))
            tol = 2.0 ** -8 * np.abs(w @ v) + (2.0 ** -10 + 2.0 ** -14) * (w @ np.abs(v)) + f16c
            assert (np.abs(out[0, t, h] - w @ v) <= tol).all()


@pytest.mark.parametrize("hq,hkv", [(7, 1), (10, 2), (3, 3), (9, 3), (20, 4)])
@pytest.mark.parametrize("c", [1, 5, 40])
@pytest.mark.parametrize("km", [ROW, CHANNEL])
def test_group_sizes(kvq, hq, hkv, c, km):
    """Groups of 1, 3, 5 and 7 query heads, whose tiles end inside 128 rows."""
    for d in (128, 256):
        case = ref.Case(d=d, km=km, vm=km, hq=hq, hkv=hkv, c=c, lens=(150, 77), seed=hq)
        cache = ref.Cache(case)
        s = slopes_of(hq, -0.05)
        begin, end = documents(case, (60, 111))
        check(cache, run(kvq, cache, s, begin, end), s, begin, end)


@pytest.mark.parametrize("dtype", [INT8, FP8, INT4])
@pytest.mark.parametrize("d,c,hq,hkv", [(64, 4, 4, 1), (128, 3, 8, 4), (128, 6, 8, 2), (128, 40, 8, 2), (256, 2, 8, 2),
                                        (256, 8, 12, 2), (256, 50, 12, 2), (576, 2, 8, 1), (576, 9, 8, 1)])
def test_lse_of_a_per_channel_scale(kvq, dtype, d, c, hq, hkv):
    """lse is fp32-accurate with a per-channel K scale too: the two-part operand
    leaves 2^-22 of sum |q k| (2^-11 with one part), on every layout; without an
    lse the one-part kernels give the same output within its bound."""
    if d == 576 and dtype == INT4:
        pytest.skip("576-channel rows are 8-bit")
    case = ref.Case(dtype=dtype, km=CHANNEL, vm=CHANNEL, d=d, c=c, hq=hq, hkv=hkv, lens=(130, 64), latent=d == 576,
                    dv=512 if d == 576 else 0)
    cache = ref.Cache(case)
    s = [0.5] * hq  # steep: few keys carry a row, so their errors do not average out
    out, lse = run(kvq, cache, s)
    r_out, r_lse, absv, f16, size = ref.attend(cache, s)
    # 2^-22 of the operand, 64 fp32 accumulations (2^-18 of their size), and a
    # few roundings of the result
    assert (np.abs(lse - r_lse) <= 2.0 ** -17 * size + 2.0 ** -20 * (1 + np.abs(r_lse))).all()
    check(cache, (out, lse), s)
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(2, hq, c, cache.width)
    ws = torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
    o2 = torch.zeros((2, c, hq, g.out_dim), dtype=torch.bfloat16, device="cuda")
    kvq.kvq_attend_masked(g, p, kvq.ScoreMask(slopes=dev(np.array(s, np.float32))), dev(cache.q).to(torch.bfloat16),
                          dev(cache.table), dev(np.array(case.lens, np.int32)), None, o2, None, ws)
    check(cache, (o2.double().cpu().numpy(), lse), s)


@pytest.mark.parametrize("c", [1, 40])
def test_tcgen05_off_and_bounds(kvq, c):
    """KVQ_DECODE_NO_TCGEN05 takes the mma.sync kernel; a max_seq_len below the
    capacity bounds the plan; the early-read flags change nothing."""
    case = ref.Case(d=128, c=c, lens=(201, 130))
    cache = ref.Cache(case, width=40)
    s = slopes_of(8)
    check(cache, run(kvq, cache, s, flags=kvq.DECODE_NO_TCGEN05), s)
    a = run(kvq, cache, s)
    b = run(kvq, cache, s, flags=kvq.DECODE_EARLY_INPUTS | kvq.DECODE_EARLY_CACHE)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    g = gpu_cache(kvq, cache)
    p = kvq.make_params(2, 8, c, cache.width, max_seq_len=201)
    ws = guarded(torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda"), "ws")
    out, lse = torch.zeros((2, c, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, c, 8), device="cuda")
    kvq.kvq_attend_masked(g, p, kvq.ScoreMask(slopes=dev(np.array(s, np.float32))), dev(cache.q).to(torch.bfloat16),
                          dev(cache.table), dev(np.array(case.lens, np.int32)), None, out, lse, ws)
    check(cache, (out.double().cpu().numpy(), lse.double().cpu().numpy()), s)
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("d,c,km", [(64, 1, ROW), (128, 4, CHANNEL), (128, 40, ROW), (256, 50, CHANNEL), (256, 70, ROW)])
def test_captured_and_on_two_streams(kvq, d, c, km):
    """Two calls with workspaces of their own, on two streams at once and
    captured into graphs that replay on two streams: the same bits as one call
    at a time."""
    calls = []
    for seed in (1, 2):
        case = ref.Case(d=d, km=km, vm=km, c=c, lens=(900, 150, 411), seed=seed)
        cache = ref.Cache(case)
        s = slopes_of(8)
        want = run(kvq, cache, s)
        check(cache, want, s)
        g = gpu_cache(kvq, cache)
        p = kvq.make_params(3, 8, c, cache.width)
        ws = torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
        out = torch.zeros((3, c, 8, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((3, c, 8), device="cuda")
        args = (g, p, kvq.ScoreMask(slopes=dev(np.array(s, np.float32))), dev(cache.q).to(torch.bfloat16),
                dev(cache.table), dev(np.array(case.lens, np.int32)), None, out, lse, ws)
        calls.append((args, want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        for args, want, _ in calls:
            assert np.array_equal(args[7].double().cpu().numpy(), want[0])
            assert np.array_equal(args[8].double().cpu().numpy(), want[1])
            args[7].zero_()
            args[8].zero_()
        torch.cuda.synchronize()

    for _ in range(4):
        for args, _, st in calls:
            kvq.kvq_attend_masked(*args, stream=st)
    same()
    graphs = []
    for args, _, st in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            kvq.kvq_attend_masked(*args)
        graphs.append((gr, st))
    for _ in range(4):
        for gr, st in graphs:
            with torch.cuda.stream(st):
                gr.replay()
    same()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("d,c", [(64, 1), (128, 40), (256, 3)])
def test_bad_pages_and_lengths_are_flagged(kvq, d, c):
    """A block id outside the pool, or a length outside the capacity, sets the
    device error; the other sequences' rows are right."""
    case = ref.Case(d=d, c=c, lens=(100, 90, 170))
    cache = ref.Cache(case)
    want = run(kvq, cache)
    good = cache.table.copy()
    g = gpu_cache(kvq, cache)
    for bad in (cache.nb, -1, 2 ** 31 - 1):
        table = good.copy()
        table[1, 2] = bad
        for lens, err in (((100, 90, 170), kvq.DEVERR_BLOCK_ID), ((100, -3, 170), kvq.DEVERR_SEQ_LEN)):
            p = kvq.make_params(3, 8, c, cache.width)
            ws = torch.zeros(kvq.kvq_attend_masked_workspace_size(g, p) // 4, dtype=torch.int32, device="cuda")
            out = torch.zeros((3, c, 8, d), dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros((3, c, 8), device="cuda")
            kvq.kvq_attend_masked(g, p, None, dev(cache.q).to(torch.bfloat16), dev(table),
                                  dev(np.array(lens, np.int32)), None, out, lse, ws)
            assert kvq.kvq_get_device_error() == err
            o = out.double().cpu().numpy()
            assert np.allclose(o[[0, 2]], want[0][[0, 2]], rtol=2.0 ** -7, atol=2.0 ** -7)
