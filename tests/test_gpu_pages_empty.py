"""kvq_pages_step for a batch of no sequences."""
import numpy as np
import pytest

import step_ref
from test_gpu_pages import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


@pytest.mark.parametrize("room", [1, 40, 5000])
@pytest.mark.parametrize("count", [0, 3, 6])
@pytest.mark.parametrize("in_place", [False, True])
def test_no_sequences(kvq, room, count, in_place):
    """The pool's count is passed on, the prefix sums are one 0, the map is empty."""
    ref = step_ref.Pages(16, 4, 6, room)
    none = np.zeros(0, np.int32)
    x = none, none, none, np.zeros((0, 4), np.int32), np.arange(6, dtype=np.int32), count
    check(run(kvq, ref, *x, in_place=in_place), ref.step(*x))
    check(run(kvq, ref, *x, parents=np.zeros((0, 3), np.int32)), ref.step(*x, parents=np.zeros((0, 3), np.int32)))


def test_no_sequences_and_no_tokens(kvq):
    """Nothing to do, and nothing is written."""
    ref = step_ref.Pages(16, 4, 6, 0)
    none = np.zeros(0, np.int32)
    got = run(kvq, ref, none, none, none, np.zeros((0, 4), np.int32), np.arange(6, dtype=np.int32), 4)
    assert list(got[1]) == list(range(6)) and got[2] == 77 and list(got[4]) == [77] and got[7] == 0
