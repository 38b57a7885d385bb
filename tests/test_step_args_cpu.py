"""The prompt, draft-tree and page calls refuse bad shapes, pointers and
overlapping buffers on the host, before any launch."""
import ctypes

import pytest

FAKE = 0x7F0000000000  # addresses that are never dereferenced on the host
B, T, HKV, BS, WIDTH, NB, ROOM = 3, 12, 2, 16, 8, 64, 40


@pytest.fixture(scope="module")
def kvq():
    from decode_attention_quantized_gb300 import build, kvq
    build.build()
    kvq.load()
    return kvq


def places(sizes):
    return {n: FAKE + (i << 24) for i, n in enumerate(sizes)}


# ------------------------------------------------------------------- pages

PAGES = {"held": 4 * B, "start": 4 * B, "new": 4 * B, "parents": 4 * B * T, "table": 4 * B * WIDTH, "free": 4 * NB,
         "count": 4, "lens": 4 * B, "left": 4, "cu": 4 * B + 4, "slots": 8 * ROOM, "positions": 8 * ROOM}
WRITTEN = ("table", "free", "lens", "left", "cu", "slots", "positions")


def pages(kvq, at, **kw):
    p = kvq.make_pages_params(**{**dict(batch=B, max_blocks_per_seq=WIDTH, num_blocks=NB, block_size=BS, max_tokens=ROOM,
                                        tree_nodes=T), **kw})
    return kvq.load().kvq_pages_step(ctypes.byref(p), *(at[n] for n in PAGES), None)


@pytest.mark.parametrize("out", WRITTEN)
@pytest.mark.parametrize("other", PAGES)
def test_pages_overlaps_are_refused(kvq, out, other):
    if out == other:
        return
    at = places(PAGES)
    tries = {at[other] + PAGES[other] - 4, at[other] - PAGES[out] + 4}
    if (out, other) not in {("lens", "held"), ("lens", "start"), ("left", "count")}:
        tries.add(at[other])
    elif out == "left":
        tries = set()
    for a in tries:
        if a % (8 if out in ("slots", "positions") else 4) == 0:
            assert pages(kvq, {**at, out: a}) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(batch=1025), 2), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1),
    (dict(block_size=8), 1), (dict(block_size=24), 1), (dict(block_size=1 << 21), 1), (dict(max_tokens=-1), 1),
    (dict(max_tokens=(1 << 30) + 1), 2), (dict(tree_nodes=0), 1), (dict(tree_nodes=257), 2),
    (dict(num_blocks=1 << 27), 1), (dict(max_blocks_per_seq=(1 << 26) + 1), 1), (dict(batch=0, max_tokens=0), 0)])
def test_pages_shapes(kvq, kw, status):
    assert pages(kvq, places(PAGES), **kw) == status


@pytest.mark.parametrize("name", PAGES)
def test_pages_pointers(kvq, name):
    at = places(PAGES)
    if name not in ("start", "parents"):
        assert pages(kvq, {**at, name: None}) == 1
    assert pages(kvq, {**at, name: at[name] + 2}) == 1
    if name in ("slots", "positions"):
        assert pages(kvq, {**at, name: at[name] + 4}) == 1


# ------------------------------------------------------------------- trees

def cache(kvq, at=None, **kw):
    at = at or {}
    f = dict(dtype=kvq.INT8, k_mode=kvq.PER_ROW, v_mode=kvq.PER_ROW, num_blocks=NB, block_size=BS, num_kv_heads=HKV,
             head_dim=64, k_codes=at.get("k_codes", FAKE), v_codes=at.get("v_codes", FAKE),
             k_scale=at.get("k_scale", FAKE), v_scale=at.get("v_scale", FAKE))
    return kvq.CacheDesc(**{**f, **kw})


ACCEPT = {"parents": 4 * B * T, "nodes": 4 * B, "drafts": 8 * B * T, "chosen": 8 * B * T, "table": 4 * B * WIDTH,
          "seq": 4 * B, "path": 4 * B * T, "accepted": 4 * B, "new": 4 * B, "next": 8 * B, "mass": 4 * NB * HKV * BS,
          "k_codes": NB * HKV * BS * 64, "v_codes": NB * HKV * BS * 64, "k_scale": 4 * NB * HKV * BS,
          "v_scale": 4 * NB * HKV * BS}
ARGS = ("drafts", "chosen", "table", "seq", "path", "accepted", "new", "next", "mass")


def accept(kvq, at, batch=B, nodes=T, width=WIDTH, top=0, **kw):
    p = kvq.make_params(batch, 4, nodes, width, max_seq_len=top)
    c, t = cache(kvq, at, **kw), kvq.TreeDesc(at["parents"], at["nodes"])
    return kvq.load().kvq_tree_accept(ctypes.byref(c), ctypes.byref(p), ctypes.byref(t), *(at[n] for n in ARGS), None)


@pytest.mark.parametrize("out", ["path", "accepted", "new", "next", "mass", "k_codes", "v_codes", "k_scale", "v_scale"])
@pytest.mark.parametrize("other", ACCEPT)
def test_accept_overlaps_are_refused(kvq, out, other):
    if out == other:
        return
    at = places(ACCEPT)
    align = 16 if "codes" in out or "scale" in out else (8 if out == "next" else 4)
    for a in {at[other], at[other] + ACCEPT[other] - align, at[other] - ACCEPT[out] + align}:
        a -= a % align
        if a + ACCEPT[out] > at[other] and a < at[other] + ACCEPT[other]:
            assert accept(kvq, {**at, out: a}) == 1


@pytest.mark.parametrize("kw,status", [(dict(batch=-1), 1), (dict(batch=1025), 2), (dict(nodes=0), 1), (dict(nodes=257), 2),
                                       (dict(width=0), 1), (dict(top=-1), 1), (dict(batch=0), 0), (dict(width=1 << 27), 1),
                                       (dict(head_dim=96), 2), (dict(num_kv_heads=70000), 2)])
def test_accept_shapes(kvq, kw, status):
    assert accept(kvq, places(ACCEPT), **kw) == status


@pytest.mark.parametrize("name", ARGS + ("parents", "nodes"))
def test_accept_pointers(kvq, name):
    at = places(ACCEPT)
    if name not in ("mass", "nodes"):
        assert accept(kvq, {**at, name: None}) == 1
    assert accept(kvq, {**at, name: at[name] + 2}) == 1


def attend_tree(kvq, batch=B, nodes=T, q=FAKE, parents=FAKE, num_nodes=None, table=FAKE, seq=FAKE, out=FAKE + (1 << 30),
                ws=FAKE, nbytes=1 << 30, hq=4, flags=0, tree=True, **kw):
    p = kvq.make_params(batch, hq, nodes, WIDTH, flags=flags)
    c, t = cache(kvq, **kw), kvq.TreeDesc(parents, num_nodes)
    return kvq.load().kvq_attend_tree(ctypes.byref(c), ctypes.byref(p), ctypes.byref(t) if tree else None, q, table, seq,
                                      None, out, None, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(batch=1025), 2), (dict(nodes=0), 1), (dict(nodes=257), 2), (dict(hq=5), 1), (dict(hq=18), 2),
    (dict(parents=None), 1), (dict(parents=FAKE + 2), 1), (dict(num_nodes=FAKE + 1), 1), (dict(tree=False), 1),
    (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(out=None), 1), (dict(out=FAKE), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 16), 1), (dict(table=None), 1), (dict(seq=None), 1), (dict(flags=8), 1), (dict(batch=0), 0)])
def test_attend_tree_refusals(kvq, kw, status):
    assert attend_tree(kvq, **kw) == status


# ------------------------------------------------------------------ prompts

N, HQ = 100, 4
PROMPT = {"q": 2 * N * HQ * 64, "k": 2 * N * HKV * 64, "v": 2 * N * HKV * 64, "cu": 4 * B + 4, "sink": 4 * HQ,
          "out": 2 * N * HQ * 64, "lse": 4 * N * HQ, "ws": 1 << 20}


def prompt(kvq, at, nbytes=1 << 20, strides=(0, 0, 0), **kw):
    f = dict(batch=B, total_tokens=N, num_q_heads=HQ, num_kv_heads=HKV, head_dim=64, max_seq_len=0, sm_scale=0.0,
             softcap=0.0, window=0)
    f.update(kw)
    p = kvq.PromptParams(**f, q_stride=strides[0], k_stride=strides[1], v_stride=strides[2])
    return kvq.load().kvq_attend_prompt(ctypes.byref(p), *(at[n] for n in PROMPT), nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(batch=1025), 2), (dict(total_tokens=-1), 1), (dict(num_q_heads=5), 1), (dict(num_q_heads=18), 2),
    (dict(num_kv_heads=0), 1), (dict(head_dim=96), 2), (dict(head_dim=576), 2), (dict(max_seq_len=-1), 1),
    (dict(window=-1), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(sm_scale=float("inf")), 1),
    (dict(strides=(HQ * 64 - 8, 0, 0)), 1), (dict(strides=(0, HKV * 64 + 4, 0)), 1), (dict(strides=(0, 0, -8)), 1),
    (dict(nbytes=0), 3), (dict(batch=0), 0), (dict(total_tokens=0), 0)])
def test_prompt_refusals(kvq, kw, status):
    assert prompt(kvq, places(PROMPT), **kw) == status


@pytest.mark.parametrize("name", PROMPT)
def test_prompt_pointers(kvq, name):
    at = places(PROMPT)
    if name not in ("sink", "lse"):
        assert prompt(kvq, {**at, name: None}) == 1
    assert prompt(kvq, {**at, name: at[name] + 2}) == 1


@pytest.mark.parametrize("out", ["out", "lse"])
@pytest.mark.parametrize("other", ["q", "k", "v", "cu", "sink", "out", "lse", "ws"])
def test_prompt_overlaps_are_refused(kvq, out, other):
    if out == other:
        return
    at = places(PROMPT)
    for a in {at[other], at[other] - PROMPT[out] + 16}:
        assert prompt(kvq, {**at, out: a}) == 1


def test_prompt_workspace_size(kvq):
    n = ctypes.c_size_t(0)
    p = kvq.make_prompt_params(B, N, HQ, HKV, 64)
    assert kvq.load().kvq_attend_prompt_workspace_size(ctypes.byref(p), None) == 1
    assert kvq.load().kvq_attend_prompt_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    p.head_dim = 80
    assert kvq.load().kvq_attend_prompt_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 2
