"""Attention of packed prompts (kvq_attend_prompt) against its 64-bit form.

Tolerances, per output channel, with A = sum p |v| (after the sink): bf16
rounding of the result, 2^-8 of it; the weights enter the product with V as
bf16, 2^-8 of A; fp32 sums of at most 2^14 weights and products, 2^-10 of A at
the most (one rounding of 2^-24 a term); a logit is off by at most 2^-15 of
sum |q k| (256 fp32 additions of partial sums up to that) and 2^-15 under a
cap (its tanh is 4e-7 of 50 off), which moves the result by twice that times A."""
import numpy as np
import pytest
import torch

from guard import guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def inputs(lens, hq, hkv, d, seed=0, fused=False, before=0, behind=0, amp=1.0):
    """q, k, v of the packed sequences, `before` and `behind` rows of NaN around
    them, and cu_seqlens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = before + sum(lens) + behind
    x = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda")
    x[:, :hq] *= amp
    x[:before] = float("nan")
    x[n - behind:] = float("nan")
    x = x.to(torch.bfloat16)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        parts = tuple(t.contiguous() for t in parts)
    cu = torch.tensor(np.cumsum([before] + list(lens)), dtype=torch.int32, device="cuda")
    return (*parts, cu)


def run(kvq, q, k, v, cu, *, cap=0.0, window=0, sink=None, lse=True, max_seq_len=0, sm_scale=0.0, err=0, out=None):
    N, hq, d = q.shape
    p = kvq.make_prompt_params(cu.numel() - 1, N, hq, k.shape[1], d, max_seq_len=max_seq_len, softcap=cap,
                               window=window, sm_scale=sm_scale)
    ws = guarded(torch.full((kvq.kvq_attend_prompt_workspace_size(p) // 4,), -1, dtype=torch.int32, device="cuda"), "ws")
    out = guarded(torch.full((N, hq, d), 7.0, dtype=torch.bfloat16, device="cuda"), "out")
    l = guarded(torch.full((N, hq), 7.0, device="cuda"), "lse") if lse else None
    kvq.kvq_attend_prompt(p, q, k, v, cu, sink, out, l, ws)
    assert kvq.kvq_get_device_error() == err
    return out, l


def check(q, k, v, cu, got, *, cap=0.0, window=0, sink=None, sm_scale=0.0, skip=()):
    """Rows of no sequence, and of the sequences in `skip`, keep their 7."""
    out, lse = got
    N, hq, d = q.shape
    G, bounds = hq // k.shape[1], cu.tolist()
    scale = sm_scale or d ** -0.5
    touched = torch.zeros(N, dtype=torch.bool, device="cuda")
    for b, (s0, s1) in enumerate(zip(bounds, bounds[1:])):
        if b in skip or s1 <= s0:
            continue
        touched[s0:s1] = True
        far = torch.arange(s1 - s0, device="cuda")[:, None] - torch.arange(s1 - s0, device="cuda")
        hidden = (far < 0) | (far >= window) if window else far < 0
        for h in range(hq):
            qq, kk, vv = q[s0:s1, h].double(), k[s0:s1, h // G].double(), v[s0:s1, h // G].double()
            x = qq @ kk.T * scale
            ds = 2.0 ** -15 * (qq.abs() @ kk.abs().T * scale).masked_fill(hidden, 0).amax(1) + 2.0 ** -19
            if cap:
                x = cap * torch.tanh(x / cap)
                ds = ds + 2.0 ** -15
            x = x.masked_fill(hidden, -torch.inf)
            r_lse = torch.logsumexp(x, 1)
            p = torch.exp(x - r_lse[:, None])
            if sink is not None:
                p = p * torch.sigmoid(r_lse - sink[h].double())[:, None]
            r, A = p @ vv, p @ vv.abs()
            tol = 2.0 ** -8 * r.abs() + (2.0 ** -8 + 2.0 ** -10 + 2 * ds[:, None]) * A + 1e-30
            e = (out[s0:s1, h].double() - r).abs() / tol
            assert torch.isfinite(e).all() and e.max() <= 1, f"sequence {b} head {h}: {e.max():.2f} times its bound"
            if lse is not None:
                e = (lse[s0:s1, h].double() - r_lse).abs() - (ds + 2.0 ** -20 * (1 + r_lse.abs()))
                assert e.max() <= 0, f"lse off by {e.max():.2e} more than its bound"
    assert (out[~touched] == 7).all()
    if lse is not None:
        assert (lse[~touched] == 7).all()


SHAPES = [(4, 1, 64), (8, 2, 128), (6, 1, 256), (24, 4, 128), (8, 1, 128), (3, 3, 64), (7, 1, 128), (10, 2, 256), (2, 1, 64)]
LENS = [(1,), (2, 1, 77), (128,), (129, 0, 31), (255, 257), (16, 17, 15, 1, 33), (700,), (64, 513, 0)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lens", LENS)
def test_shapes_and_lengths(kvq, hq, hkv, d, lens):
    x = inputs(lens, hq, hkv, d, seed=sum(lens) + hq)
    check(*x, run(kvq, *x))


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 2, 128), (6, 1, 256), (5, 1, 128)])
@pytest.mark.parametrize("window", [1, 2, 31, 128, 129, 300])
@pytest.mark.parametrize("cap", [0.0, 50.0])
def test_windows_caps_and_sinks(kvq, hq, hkv, d, window, cap):
    x = inputs((333, 1, 140, window), hq, hkv, d, seed=window, fused=True, amp=4.0)
    sink = torch.linspace(-1, 3, hq, device="cuda")
    check(*x, run(kvq, *x, cap=cap, window=window, sink=sink), cap=cap, window=window, sink=sink)


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (32, 8, 128), (24, 4, 256)])
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_long_prompts(kvq, hq, hkv, d, cap):
    x = inputs((2500, 1100), hq, hkv, d, seed=d)
    check(*x, run(kvq, *x, cap=cap), cap=cap)
    check(*x, run(kvq, *x, cap=cap, window=1000, lse=False), cap=cap, window=1000)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_scores_and_given_scales(kvq, d):
    """Weights of one key only, maxima that grow along a row, a scale of one."""
    q, k, v, cu = inputs((400,), 4, 2, d, amp=8.0)
    ramp = torch.linspace(0.01, 3.0, 400, device="cuda")[:, None, None]
    k = (k.float() * ramp).to(torch.bfloat16)
    check(q, k, v, cu, run(kvq, q, k, v, cu, sm_scale=0.3), sm_scale=0.3)
    check(q, -k, v, cu, run(kvq, q, -k, v, cu))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_no_sequence_may_hold_anything(kvq, d):
    x = inputs((130, 40, 1), 8, 2, d, before=5, behind=70)
    check(*x, run(kvq, *x))
    x = inputs((130, 40, 1), 8, 2, d, before=3, behind=1, fused=True)
    check(*x, run(kvq, *x, window=50), window=50)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_sequence_or_query_stays_alone(kvq, d, bad):
    """The rows of one sequence hold NaN or infinities: the others do not show
    it, next to it or not.  A bad query is its own token's alone."""
    lens = (70, 60, 130, 9)
    q, k, v, cu = inputs(lens, 8, 2, d)
    for t in (q, k, v):
        t[70:130] = bad
    out, lse = run(kvq, q, k, v, cu)
    out[70:130], lse[70:130] = 7.0, 7.0
    check(q, k, v, cu, (out, lse), skip=(1,))
    q, k, v, cu = inputs(lens, 8, 2, d)
    good = run(kvq, q, k, v, cu)
    q[33, 3] = bad
    out, lse = run(kvq, q, k, v, cu)
    rest = torch.ones((sum(lens), 8), dtype=torch.bool, device="cuda")
    rest[33, 3] = False
    assert torch.equal(out[rest], good[0][rest]) and torch.equal(lse[rest], good[1][rest])


def test_bounds_that_descend_or_leave_the_rows_are_flagged(kvq):
    q, k, v, _ = inputs((50, 60, 70, 20), 4, 2, 128)
    bounds = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = bounds(0, 50, 300, 300, 300)
    check(q, k, v, bounds(0, 50), run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN))
    cu = bounds(-7, 50, 110, 180, 2 ** 31 - 1)
    check(q, k, v, bounds(50, 110, 180), run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN))
    cu = bounds(0, 50, 20, 20, 90)  # 50 -> 20 descends; rows 20..89 are the last one's
    out, lse = run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN)
    assert torch.isfinite(out.float()).all() and (out[90:] == 7).all()
    cu = bounds(0, 50, 110, 180, 200)
    check(q, k, v, cu, run(kvq, q, k, v, cu, max_seq_len=60, err=kvq.DEVERR_SEQ_LEN), skip=(2,))


def test_many_short_sequences(kvq):
    r = np.random.default_rng(2)
    lens = tuple(int(x) for x in r.integers(0, 9, 1024))
    x = inputs(lens, 8, 2, 128, seed=9)
    out, lse = run(kvq, *x)
    for lo in (0, 500, 1000):  # three runs of them against the 64-bit form
        part = x[3][lo:lo + 25]
        o, l = torch.full_like(out, 7), torch.full_like(lse, 7)
        o[part[0]:part[-1]], l[part[0]:part[-1]] = out[part[0]:part[-1]], lse[part[0]:part[-1]]
        check(*x[:3], part, (o, l))
    assert not (out == 7).all(-1).any()


def test_offsets_past_32_bits(kvq):
    """150,000 tokens of 64 heads of 256 channels: 2.5 billion elements of q and out."""
    lens = (1000,) * 149 + (871,)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    N, hq, hkv, d = sum(lens), 64, 8, 256
    q = torch.empty((N, hq, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k = torch.empty((N, hkv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty((N, hkv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device="cuda")
    p = kvq.make_prompt_params(len(lens), N, hq, hkv, d)
    ws = torch.empty(kvq.kvq_attend_prompt_workspace_size(p) // 4, dtype=torch.int32, device="cuda")
    out = torch.full((N, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvq.kvq_attend_prompt(p, q, k, v, cu, None, out, None, ws)
    assert kvq.kvq_get_device_error() == 0
    s = N - 871
    tail = torch.tensor([0, 871], dtype=torch.int32, device="cuda")
    check(q[s:, :8], k[s:, :1], v[s:, :1], tail, (out[s:, :8], None))
    check(q[s:, 56:], k[s:, 7:], v[s:, 7:], tail, (out[s:, 56:], None))


def test_repeated_calls_streams_and_graphs_give_the_same_bits(kvq):
    q, k, v, cu = inputs((300, 41, 129), 24, 4, 128)
    first = run(kvq, q, k, v, cu)
    for _ in range(3):
        again = run(kvq, q, k, v, cu)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(kvq, q, k, v, cu)
    assert torch.equal(first[0], again[0])
    p = kvq.make_prompt_params(3, 470, 24, 4, 128)
    ws = torch.empty(kvq.kvq_attend_prompt_workspace_size(p) // 4, dtype=torch.int32, device="cuda")
    bounds = torch.tensor([0, 0, 0, 470], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(first[0], 7), torch.full_like(first[1], 7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_attend_prompt(p, q, k, v, bounds, None, out, lse, ws)
    graph.replay()
    bounds.copy_(cu)  # other lengths, the same graph
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_two_streams_at_once(kvq):
    """Two calls with workspaces of their own run side by side."""
    x = [inputs((900, 300), 8, 2, 128, seed=s) for s in (1, 2)]
    want = [run(kvq, *y) for y in x]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    p = kvq.make_prompt_params(2, 1200, 8, 2, 128)
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            ws = torch.empty(kvq.kvq_attend_prompt_workspace_size(p) // 4, dtype=torch.int32, device="cuda")
            out, lse = torch.empty_like(want[i][0]), torch.empty_like(want[i][1])
            for _ in range(4):
                kvq.kvq_attend_prompt(p, *x[i], None, out, lse, ws)
            got.append((out, lse, ws))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
