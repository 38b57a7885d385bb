"""Bounds of packed prompts (kvq_attend_prompt) that descend: no row belongs to
two sequences, the others are whole, and the rest keeps what it held."""
import numpy as np
import pytest
import torch

from test_gpu_prompt import check, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


def skipped(bounds, N, top=None):
    """The sequences that are skipped: with bounds of their own that are wrong,
    or from before the end of one whose bounds are right."""
    got, end = [], 0
    for b, (s0, s1) in enumerate(zip(bounds, bounds[1:])):
        own = 0 <= s0 <= s1 <= N and s1 - s0 <= (top or N)
        if not own or s0 < end:
            got.append(b)
        if own:
            end = max(end, s1)
    return got


@pytest.mark.parametrize("bounds", [
    (0, 50, 20, 20, 90), (0, 50, 20, 90, 200), (100, 180, 0, 60, 200), (0, 200, 0, 200, 0, 200), (0, 150, 60, 160, 150, 200),
    (10, 300, 20, 90, 120), (0, 40, 30, 35, 33, 40, 38, 60, 55, 200), (0, -5, 30, 200), (60, 60, 50, 70, 70, 65, 65, 90)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_descending_bounds(kvq, bounds, d):
    q, k, v, _ = inputs((200,), 4, 2, d, seed=1)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    check(q, k, v, cu, run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN), skip=skipped(bounds, 200))


@pytest.mark.parametrize("B", [31, 33, 64, 65, 300, 1024])
def test_descents_among_many_sequences(kvq, B):
    """More sequences than a warp, than the unplanned launch takes, and the most."""
    r = np.random.default_rng(B)
    q, k, v, _ = inputs((2000,), 4, 2, 64, seed=B)
    bounds = np.sort(r.integers(0, 2001, B + 1))
    for i in r.choice(B, max(2, B // 50), replace=False):
        bounds[i] = max(0, bounds[i] - int(r.integers(1, 400)))
    bounds = [int(x) for x in bounds]
    skip = skipped(bounds, 2000)
    assert 0 < len(skip) < B
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    check(q, k, v, cu, run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN), skip=skip)


def test_the_whole_pack_many_times_over(kvq):
    """Bounds that go back and forth over all rows: one sequence's work."""
    q, k, v, _ = inputs((6000,), 8, 2, 128, seed=3)
    cu = torch.tensor([0, 6000] * 500, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 6000], dtype=torch.int32, device="cuda")
    got, want = run(kvq, q, k, v, cu, err=kvq.DEVERR_SEQ_LEN), run(kvq, q, k, v, good)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
