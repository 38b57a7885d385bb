"""Masked attention and key mass at the edges of what their arguments allow,
against the 64-bit forms of score_ref."""
import dataclasses

import numpy as np
import pytest
import torch

import score_ref as ref
from guard import guarded
from test_gpu_masked import CASES, check, dev, gpu_cache, run, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import kvq
    kvq.load()
    return kvq


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
