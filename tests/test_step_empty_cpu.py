"""The tree and prompt calls do nothing for a batch of no sequences, whose
tensors have no address."""
import ctypes

import pytest

from test_step_args_cpu import FAKE, WIDTH, cache, kvq  # noqa: F401 (the fixture)


@pytest.mark.parametrize("parents", [None, FAKE])
def test_no_trees(kvq, parents):  # noqa: F811
    c, t = cache(kvq), kvq.TreeDesc(parents, None)
    p = kvq.make_params(0, 4, 12, WIDTH)
    assert kvq.load().kvq_attend_tree(ctypes.byref(c), ctypes.byref(p), ctypes.byref(t), *[None] * 6, None, 0, None) == 0
    assert kvq.load().kvq_tree_accept(ctypes.byref(c), ctypes.byref(p), ctypes.byref(t), *[None] * 10) == 0
    p.batch = 1
    if parents is None:
        assert kvq.load().kvq_tree_accept(ctypes.byref(c), ctypes.byref(p), ctypes.byref(t), *[None] * 10) == 1


def test_no_prompts(kvq):  # noqa: F811
    p = kvq.make_prompt_params(0, 0, 4, 2, 64)
    assert kvq.load().kvq_attend_prompt(ctypes.byref(p), *[None] * 8, 0, None) == 0
