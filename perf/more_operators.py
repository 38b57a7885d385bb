"""Operators of a serving step around the quantized paged cache, as their users
call them, and their plain forms.

  prompt  causal attention of whole prompts, packed, over the bf16 q, k, v in hand
  tree    attention of drafted token trees over the quantized paged cache
  accept  the accepted path of each tree and the move of its cache rows
  pages   block tables, slot map, positions and free list from request lengths

A case is a dict of plain values; lengths, node counts and page counts follow
from the case alone, all values from the seed."""
import math
import random

import numpy as np
import torch

own = False

INT8, FP8, INT4 = 1, 2, 3
ROW, TENSOR, CHANNEL = 1, 2, 3
QMAX = {INT8: 127.0, FP8: 448.0, INT4: 7.0}
VOCAB = 32000

# cache kinds of the repository's workloads: types, scale modes, heads, block
# size, softcap, head sink, and (block 256) block ids in order or shuffled
KINDS = {
    "tiny": dict(dtype=INT8, km=ROW, vm=ROW, hq=4, hkv=1, d=64, block=256, cap=0.0, sink=False),
    "gqa": dict(dtype=INT8, km=ROW, vm=ROW, hq=24, hkv=4, d=256, block=256, cap=0.0, sink=False),
    "paged": dict(dtype=FP8, km=TENSOR, vm=TENSOR, hq=32, hkv=8, d=128, block=16, cap=50.0, sink=False),
    "spec": dict(dtype=INT4, km=CHANNEL, vm=CHANNEL, hq=24, hkv=4, d=256, block=32, cap=0.0, sink=False),
    "mixed": dict(dtype=INT8, km=CHANNEL, vm=TENSOR, hq=64, hkv=8, d=128, block=256, cap=0.0, sink=True),
}


def listed():
    return [
        # one short question to a small model: latency
        dict(name="prompt_short", op="prompt", kind="tiny", batch=1, ctx=77, ragged=False, window=0, fused=False),
        # a batch of unequal prompts of a capped model
        dict(name="prompt_packed_ragged", op="prompt", kind="paged", batch=16, ctx=4096, ragged=True, window=0,
             fused=False),
        # one long document
        dict(name="prompt_long", op="prompt", kind="mixed", batch=1, ctx=16384, ragged=False, window=0, fused=False),
        # prompts of an odd length in a windowed layer, q, k, v as slices of one projection
        dict(name="prompt_window_fused", op="prompt", kind="gqa", batch=3, ctx=8191, ragged=True, window=1024,
             fused=True),
        # a few drafts over a short conversation of a small model: latency
        dict(name="tree_short", op="tree", kind="tiny", batch=1, nodes=7, ctx=2048, ragged=False, window=0),
        # sixteen drafts over one long conversation
        dict(name="tree_long", op="tree", kind="gqa", batch=1, nodes=16, ctx=131072, ragged=False, window=0),
        # wide trees over a few conversations, 4-bit cache
        dict(name="tree_wide", op="tree", kind="spec", batch=4, nodes=32, ctx=32768, ragged=False, window=0),
        # a serving batch of unequal lengths and trees in small shuffled pages
        dict(name="tree_ragged", op="tree", kind="paged", batch=16, nodes=13, ctx=32768, ragged=True, window=0),
        # one conversation after a step of eight drafts
        dict(name="accept_one", op="accept", kind="gqa", batch=1, nodes=8, ctx=4096, ragged=False),
        # a large batch after a step of wide trees
        dict(name="accept_batch", op="accept", kind="mixed", batch=64, nodes=64, ctx=1024, ragged=True),
        # a serving batch between two decode steps
        dict(name="pages_decode", op="pages", batch=64, block=16, ctx=8192, mix="decode", nodes=0, short=False),
        # a full batch that takes in new prompts and lets finished ones go
        dict(name="pages_prompts", op="pages", batch=1024, block=16, ctx=8192, mix="prompts", nodes=0, short=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "accept", "pages"])
    if op == "prompt":
        batch = _log(rng, 1, 32)
        return dict(op=op, kind=rng.choice(["tiny", "gqa", "paged", "mixed"]), batch=batch,
                    ctx=_log(rng, 1, int(14000 / math.sqrt(batch))), ragged=rng.random() < 0.5,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), fused=rng.random() < 0.5)
    if op == "tree":
        batch = _log(rng, 1, 16)
        nodes = _log(rng, 1, 64)
        return dict(op=op, kind=rng.choice(["tiny", "gqa", "paged", "spec", "mixed"]), batch=batch, nodes=nodes,
                    ctx=nodes + _log(rng, 1, (262144 if nodes <= 16 else 100000) // batch),
                    ragged=rng.random() < 0.5, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    if op == "accept":
        batch = _log(rng, 1, 64)
        nodes = _log(rng, 1, 64)
        return dict(op=op, kind=rng.choice(["tiny", "gqa", "paged", "mixed"]), batch=batch, nodes=nodes,
                    ctx=nodes + _log(rng, 1, 65536 // batch), ragged=rng.random() < 0.5)
    batch = _log(rng, 1, 1024)
    mix = rng.choice(["decode", "draft", "prompts"])
    return dict(op=op, batch=batch, block=rng.choice([16, 32, 256]), ctx=_log(rng, 64, 8192), mix=mix,
                nodes=_log(rng, 2, 64) if mix == "draft" else 0, short=rng.random() < 0.25)


# ------------------------------------------------- what follows from a case

def _rng(case, what):
    return random.Random(what + " %s" % sorted((k, str(v)) for k, v in case.items() if k != "name"))


def _lens(case):
    """Sequence lengths: `ctx` for all, or from 1/16 of it to all of it (the
    first sequence has the whole); never shorter than a tree of drafts."""
    r, lo = _rng(case, "lengths"), max(case.get("nodes", 1), case["ctx"] // 16, 1)
    if not case["ragged"]:
        return [case["ctx"]] * case["batch"]
    return [case["ctx"]] + [r.randint(lo, max(lo, case["ctx"])) for _ in range(case["batch"] - 1)]


def _nodes(case):
    """Drafted nodes of each sequence: all, or from half of them up."""
    r, T = _rng(case, "nodes"), case["nodes"]
    return [r.randint((T + 1) // 2, T) if case["ragged"] else T for _ in range(case["batch"])]


def _requests(case):
    """held, start, new of each sequence (rows whose pages it holds, rows that
    stay, rows to come), and the pool: blocks in all, free ones among them."""
    r, ctx, bs = _rng(case, "requests"), case["ctx"], case["block"]
    rows = []
    for _ in range(case["batch"]):
        held = _log(r, max(1, ctx // 16), ctx)
        if case["mix"] == "draft":
            held = max(held, case["nodes"])
            rows.append((held, held - r.randint(0, case["nodes"] - 1), r.randint(1, case["nodes"])))
            continue
        kind = r.random() if case["mix"] == "prompts" else 1.0
        if kind < 0.25:
            rows.append((0, 0, _log(r, 1, ctx)))
        elif kind < 0.5:
            rows.append((held, 0, 0))
        else:
            rows.append((held, held, 1))
    up = lambda n: -(-n // bs)  # noqa: E731
    taken = sum(up(h) for h, _, _ in rows)
    grow = sum(max(0, up(s + n) - up(h)) for h, s, n in rows)
    back = sum(max(0, up(h) - up(s + n)) for h, s, n in rows)
    free = max(0, (6 * grow // 10 if case["short"] else grow + 8) - back)
    return rows, taken + free, free


def _granted(case):
    """Which sequences get their pages: in order, while the pool suffices."""
    rows, _, free = _requests(case)
    up = lambda n: -(-n // case["block"])  # noqa: E731
    have = free + sum(max(0, up(h) - up(s + n)) for h, s, n in rows)
    got, asked = [], 0
    for h, s, n in rows:
        more = max(0, up(s + n) - up(h))
        asked += more
        got.append(more == 0 or asked <= have)
    return got


def _pairs(case):
    """Visible (query token, key) pairs of one query head of a prompt."""
    W, n = case["window"], 0
    for L in _lens(case):
        n += L * (L + 1) // 2 if W == 0 or W >= L else W * (W + 1) // 2 + (L - W) * W
    return n


def _row_bytes(k):
    code = k["d"] // 2 if k["dtype"] == INT4 else k["d"]
    return sum(code + (4 if m == ROW else 0) for m in (k["km"], k["vm"]))


def work(case):
    if case["op"] == "pages":
        rows, _, _ = _requests(case)
        up = lambda n: -(-n // case["block"])  # noqa: E731
        ok = _granted(case)
        tokens = _room(case)
        named = sum(abs(up(s + n) - up(h)) for (h, s, n), g in zip(rows, ok) if g)
        drafts = 4 * sum(n for _, _, n in rows) if case["nodes"] else 0
        return dict(bytes=16 * tokens + 8 * named + 20 * case["batch"] + drafts, flops=0)
    k, lens = KINDS[case["kind"]], _lens(case)
    if case["op"] == "prompt":
        n = sum(lens)
        return dict(bytes=2 * n * k["d"] * (2 * k["hq"] + 2 * k["hkv"]) + 4 * n * k["hq"],
                    flops=4 * k["d"] * k["hq"] * _pairs(case))
    tables = 4 * sum((L + k["block"] - 1) // k["block"] for L in lens) + 8 * len(lens)
    if case["op"] == "tree":
        W, nodes = case["window"], _nodes(case)
        keys = sum(min(L, W + T) if W else L for L, T in zip(lens, nodes))
        pairs = sum(T * ((min(L - T, W) if W else L - T) + 1) for L, T in zip(lens, nodes)) * k["hq"]
        rows = case["batch"] * case["nodes"] * k["hq"]
        return dict(bytes=keys * k["hkv"] * _row_bytes(k) + rows * (4 * k["d"] + 4) + tables, flops=4 * k["d"] * pairs)
    # about five rows of a path move; the trees are read whole
    T = sum(_nodes(case))
    return dict(bytes=min(5 * case["batch"], T) * k["hkv"] * 2 * (_row_bytes(k) + 4) + 20 * T + tables, flops=0)


def _room(case):
    """Entries of the slot map: the step's tokens, rounded up as a captured
    graph's buffers are."""
    return max(64, -(-sum(n for _, _, n in _requests(case)[0]) // 64) * 64)


# ------------------------------------------------------------------ inputs

def _make_side(k, mode, blocks, g, spread):
    """Codes and scales of one side, drawn in the cache's own layout
    [blocks, Hkv, block, D]: normal values (K channels of unequal size),
    quantized as the cache holds them."""
    hkv, bs, d, dt = k["hkv"], k["block"], k["d"], k["dtype"]
    f = torch.exp(spread * torch.randn((hkv, 1, d), generator=g, device="cuda"))
    scale = torch.empty((blocks, hkv, bs), dtype=torch.float32, device="cuda") if mode == ROW else None
    codes = torch.empty((blocks, hkv, bs, d // 2 if dt == INT4 else d), dtype=torch.uint8, device="cuda")
    if mode == TENSOR:
        scale = torch.full((1,), 5.0 / QMAX[dt], device="cuda")
    if mode == CHANNEL:
        scale = (f[:, 0] * 4.5 / QMAX[dt]).contiguous()
    step = max(1, (1 << 27) // (hkv * bs * d))
    for i in range(0, blocks, step):
        x = torch.randn((min(step, blocks - i), hkv, bs, d), generator=g, device="cuda") * f
        if mode == ROW:
            s = x.abs().amax(-1) / QMAX[dt]
            scale[i:i + step] = s
            s = s[..., None]
        else:
            s = scale if mode == TENSOR else scale[:, None, :]
        c = x / s
        if dt == FP8:
            codes[i:i + step] = c.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            c = c.round().clamp(-QMAX[dt], QMAX[dt]).to(torch.int32)
            codes[i:i + step] = (c if dt == INT8 else (c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8)
    return codes, scale


def _make_tree(s, case, g):
    """Parents (one of the up to six nodes before), drafted tokens, and the
    model's choice after each node: four times of five its first child's token."""
    B, T = case["batch"], case["nodes"]
    at = torch.arange(T, device="cuda")
    r = torch.rand((B, T), generator=g, device="cuda")
    s["parents"] = (at - 1 - (r * at.clamp(max=6)).long().clamp(max=5)).clamp(min=-1).to(torch.int32)
    s["drafts"] = torch.randint(0, VOCAB, (B, T), generator=g, device="cuda")
    child = torch.full((B, T + 1), T, device="cuda")
    child.scatter_reduce_(1, torch.where(s["parents"] < 0, T, s["parents"].long()), at.expand(B, T), "amin")
    child = child[:, :T]
    other = torch.randint(0, VOCAB, (B, T), generator=g, device="cuda")
    follow = (torch.rand((B, T), generator=g, device="cuda") < 0.8) & (child < T)
    s["chosen"] = torch.where(follow, s["drafts"].gather(1, child.clamp(max=T - 1)), other)
    s["nodes"] = torch.tensor(_nodes(case), dtype=torch.int32, device="cuda") if case["ragged"] else None


def _prepare_pages(case, g):
    rows, blocks, free = _requests(case)
    B, bs = case["batch"], case["block"]
    width = max(-(-max(h, s + n) // bs) for h, s, n in rows)
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(1, width)), dtype=torch.int32, device="cuda")
    need = torch.tensor([-(-h // bs) for h, _, _ in rows], device="cuda")
    table[torch.arange(max(1, width), device="cuda") < need[:, None]] = perm[:blocks - free]
    pool = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    pool[:free] = perm[blocks - free:]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    room = _room(case)
    s = dict(case=case, table=table, pool=pool, free=ints([free]), held=ints([h for h, _, _ in rows]),
             start=ints([x for _, x, _ in rows]), new=ints([n for _, _, n in rows]), parents=None,
             lens=ints([0] * B), left=ints([0]), cu=ints([0] * (B + 1)),
             slots=torch.empty((room,), dtype=torch.int64, device="cuda"),
             positions=torch.empty((room,), dtype=torch.int64, device="cuda"))
    if case["nodes"]:
        _make_tree(s, dict(case, ragged=False), g)
    if own:
        from decode_attention_quantized_gb300 import kvq
        s["params"] = kvq.make_pages_params(B, table.shape[1], num_blocks=blocks, block_size=bs, max_tokens=room,
                                            tree_nodes=case["nodes"])
    return s


def _prepare_prompt(case, g):
    k, lens = KINDS[case["kind"]], _lens(case)
    n, hq, hkv, d = sum(lens), k["hq"], k["hkv"], k["d"]
    f = torch.exp(0.5 * torch.randn((hkv, d), generator=g, device="cuda"))
    s = dict(case=case, k=k, lens=lens)
    if case["fused"]:
        x = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda")
        x[:, hq:hq + hkv] *= f
        x = x.to(torch.bfloat16)
        s["q"], s["kn"], s["vn"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        s["q"] = torch.randn((n, hq, d), generator=g, device="cuda").to(torch.bfloat16)
        s["kn"] = (torch.randn((n, hkv, d), generator=g, device="cuda") * f).to(torch.bfloat16)
        s["vn"] = torch.randn((n, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    s["cu"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    s["sink"] = torch.randn((hq,), generator=g, device="cuda") if k["sink"] else None
    s["out"] = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((n, hq), dtype=torch.float32, device="cuda")
    if own:
        from decode_attention_quantized_gb300 import kvq
        s["params"] = kvq.make_prompt_params(len(lens), n, hq, hkv, d, max_seq_len=max(lens), softcap=k["cap"],
                                             window=case["window"])
        s["ws"] = torch.empty(kvq.kvq_attend_prompt_workspace_size(s["params"]) // 4 + 64, dtype=torch.int32,
                              device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    if case["op"] == "prompt":
        return _prepare_prompt(case, g)
    k, lens = KINDS[case["kind"]], _lens(case)
    B, T, bs = case["batch"], case["nodes"], k["block"]
    need = [(L + bs - 1) // bs for L in lens]
    blocks, width = sum(need), max(need)
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    if bs == 256:
        perm = torch.arange(blocks, dtype=torch.int32, device="cuda")
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda") < torch.tensor(need, device="cuda")[:, None]] = perm
    s = dict(case=case, k=k, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), top=max(lens))
    s["kc"], s["ks"] = _make_side(k, k["km"], blocks, g, 0.5)
    s["vc"], s["vs"] = _make_side(k, k["vm"], blocks, g, 0.0)
    _make_tree(s, case, g)
    if case["op"] == "tree":
        s["q"] = torch.randn((B, T, k["hq"], k["d"]), generator=g, device="cuda").to(torch.bfloat16)
        s["sink"] = torch.randn((k["hq"],), generator=g, device="cuda") if k["sink"] else None
        s["out"] = torch.empty((B, T, k["hq"], k["d"]), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, T, k["hq"]), dtype=torch.float32, device="cuda")
    else:
        s["path"] = torch.empty((B, T), dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["next"] = torch.empty((B,), dtype=torch.int64, device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors and workspace that a user's program keeps."""
    from decode_attention_quantized_gb300 import kvq
    case, k = s["case"], s["k"]
    one = torch.ones((1,), device="cuda")
    c = s["cache"] = kvq.QuantizedPagedCache(k["dtype"], kvq.PER_TENSOR, kvq.PER_TENSOR, 1, k["block"], k["hkv"],
                                             k["d"], k_static=one, v_static=one)
    c.num_blocks, c.k_mode, c.v_mode = s["kc"].shape[0], k["km"], k["vm"]
    c.k_codes, c.v_codes, c.k_scale, c.v_scale = s["kc"], s["vc"], s["ks"], s["vs"]
    s["params"] = kvq.make_params(case["batch"], k["hq"], case["nodes"], s["table"].shape[1], max_seq_len=s["top"],
                                  softcap=k["cap"], window=case.get("window", 0))
    s["tree"] = kvq.DraftTree(s["parents"], s["nodes"])
    if case["op"] == "tree":
        s["ws"] = torch.empty(kvq.kvq_attend_tree_workspace_size(c, s["params"]) // 4 + 64, dtype=torch.int32,
                              device="cuda")


# ------------------------------------------------------------- plain forms

def _capped(x, cap):
    return cap * torch.tanh(x / cap) if cap > 0 else x


def _softmax(x):
    """Weights and log-sum-exp of fp32 scores; rows of nothing but -inf give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t > 0, t, 1.0), (m + torch.log(t))[..., 0]


def _prompt(s):
    k, W = s["k"], s["case"]["window"]
    hkv, d, G, at = k["hkv"], k["d"], k["hq"] // k["hkv"], 0
    for L in s["lens"]:
        step = max(16, (1 << 28) // (k["hq"] * L))
        for i0 in range(0, L, step):
            i1 = min(L, i0 + step)
            j0 = max(0, i0 - W + 1) if W else 0
            q = s["q"][at + i0:at + i1].float().reshape(i1 - i0, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
            key, val = (t[at + j0:at + i1].float().transpose(0, 1) for t in (s["kn"], s["vn"]))
            x = _capped(q @ key.transpose(1, 2) / math.sqrt(d), k["cap"]).reshape(hkv, G, i1 - i0, i1 - j0)
            i = torch.arange(i0, i1, device="cuda")[:, None]
            j = torch.arange(j0, i1, device="cuda")[None]
            see = (j <= i) & (j > i - W) if W else j <= i
            p, lse = _softmax(torch.where(see, x, -math.inf))
            o = (p.reshape(hkv, -1, i1 - j0) @ val).reshape(hkv, G, i1 - i0, d)
            if s["sink"] is not None:
                o = o / (1.0 + torch.exp(s["sink"].reshape(hkv, G, 1, 1) - lse[..., None]))
            s["out"][at + i0:at + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, -1, d)
            s["lse"][at + i0:at + i1] = lse.permute(2, 0, 1).reshape(i1 - i0, -1)
        at += L
    return [s["out"], s["lse"]]


def _ancestors(parents):
    """[B, T, T] truth values: node j is i's ancestor or i itself.  A parent
    outside [0, i) makes a root."""
    B, T = parents.shape
    at = torch.arange(T, device="cuda")
    p = torch.where((parents >= 0) & (parents < at), parents.long(), T)
    a = torch.eye(T, device="cuda").expand(B, T, T).clone()
    a += torch.nn.functional.one_hot(p, T + 1)[..., :T].float()
    for _ in range(max(1, T - 1).bit_length()):
        a = (a @ a).clamp(max=1.0)
    return a > 0


def _values(s, b, codes, scale, mode):
    """fp32 values [Hkv, L, D] of sequence b's rows of one side."""
    k, n = s["k"], s["lens_host"][b]
    pages = s["table"][b, :-(-n // k["block"])].long()
    c = codes[pages].transpose(0, 1).flatten(1, 2)[:, :n]
    if k["dtype"] == INT4:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
        c = torch.where(c >= 8, c - 16, c)
    else:
        c = c.view(torch.int8 if k["dtype"] == INT8 else torch.float8_e4m3fn).float()
    if mode == ROW:
        return c * scale[pages].transpose(0, 1).flatten(1, 2)[:, :n, None]
    return c * (scale if mode == TENSOR else scale[:, None, :])


def _tree(s):
    k, case = s["k"], s["case"]
    T, W, hkv, d, G = case["nodes"], case["window"], k["hkv"], k["d"], k["hq"] // k["hkv"]
    s["lens_host"] = _lens(case)
    anc = _ancestors(s["parents"])
    depth = anc.sum(-1) - 1
    s["out"].zero_()
    s["lse"].fill_(-math.inf)
    for b, (L, n) in enumerate(zip(_lens(case), _nodes(case))):
        P = L - n
        see = torch.ones((n, L), dtype=torch.bool, device="cuda")
        see[:, P:] = anc[b, :n, :n]
        if W:
            at = torch.cat([torch.arange(P, device="cuda"), P + depth[b, :n]])
            see &= at[None] > P + depth[b, :n, None] - W
        q = s["q"][b, :n].float().reshape(n, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * n, d)
        x = q @ _values(s, b, s["kc"], s["ks"], k["km"]).transpose(1, 2) / math.sqrt(d)
        x = _capped(x, k["cap"]).reshape(hkv, G, n, L)
        p, lse = _softmax(torch.where(see, x, -math.inf))
        o = (p.reshape(hkv, G * n, L) @ _values(s, b, s["vc"], s["vs"], k["vm"])).reshape(hkv, G, n, d)
        if s["sink"] is not None:
            o = o / (1.0 + torch.exp(s["sink"].reshape(hkv, G, 1, 1) - lse[..., None]))
        s["out"][b, :n] = o.permute(2, 0, 1, 3).reshape(n, k["hq"], d)
        s["lse"][b, :n] = lse.permute(2, 0, 1).reshape(n, k["hq"])
    return [s["out"], s["lse"]]


def _accept(s):
    k, case = s["k"], s["case"]
    B, T, bs = case["batch"], case["nodes"], k["block"]
    at = torch.arange(T, device="cuda")
    n = torch.full((B,), T, device="cuda") if s["nodes"] is None else s["nodes"].long()
    parents = s["parents"].long()
    good = (parents >= 0) & (parents < at) & (at < n[:, None])
    good &= s["drafts"] == s["chosen"].gather(1, parents.clamp(0, T - 1))
    cur, live = torch.zeros((B,), dtype=torch.long, device="cuda"), n > 0
    s["path"].fill_(-1)
    count = torch.zeros((B,), dtype=torch.long, device="cuda")
    last = torch.full((B,), -1, device="cuda")
    for step in range(T):
        s["path"][:, step] = torch.where(live, cur, -1).to(torch.int32)
        count += live
        last = torch.where(live, s["chosen"].gather(1, cur[:, None])[:, 0], last)
        child = torch.where(good & (parents == cur[:, None]), at, T).amin(1)
        live = live & (child < T)
        cur = torch.where(live, child, 0)
    s["accepted"].copy_(count)
    base = s["lens"].long() - n
    s["new_lens"].copy_(base + count)
    s["next"].copy_(last)
    b, i = (s["path"] >= 0).nonzero(as_tuple=True)
    src, dst = base[b] + s["path"][b, i].long(), base[b] + i
    sb, sr, db, dr = s["table"][b, src // bs].long(), src % bs, s["table"][b, dst // bs].long(), dst % bs
    for side in [s["kc"], s["vc"]] + ([s["ks"]] if k["km"] == ROW else []) + ([s["vs"]] if k["vm"] == ROW else []):
        side[db, :, dr] = side[sb, :, sr]
    return _accepted(s)


def _accepted(s):
    kind = torch.int8 if s["k"]["dtype"] == INT8 else torch.float8_e4m3fn
    return [s["path"], s["accepted"], s["new_lens"], s["next"], s["kc"].view(kind), s["vc"].view(kind), s["ks"], s["vs"]]


def _pages(s):
    case, bs = s["case"], s["case"]["block"]
    up = lambda n: (n + bs - 1) // bs  # noqa: E731
    held, start, new = s["held"].long(), s["start"].long(), s["new"].long()
    have, want = up(held), up(start + new)
    grow, back = (want - have).clamp(min=0), (have - want).clamp(min=0)
    supply = s["free"].long() + back.sum()
    ok = (grow == 0) | (grow.cumsum(0) <= supply)
    col = torch.arange(s["table"].shape[1], device="cuda")
    freed = s["table"][(col >= want[:, None]) & (col < have[:, None])]
    before = int(s["free"])
    stack = torch.cat([s["pool"][:before], freed])
    took = torch.where(ok, grow, 0)
    n = int(took.sum())
    s["table"][(col >= have[:, None]) & (col < (have + took)[:, None])] = stack.flip(0)[:n]
    left = stack.shape[0] - n
    if left > before:
        s["pool"][before:left] = stack[before:left]
    s["left"].fill_(left)
    s["lens"].copy_(torch.where(ok, start + new, held))
    s["cu"][1:] = torch.where(ok, new, 0).cumsum(0)
    token = torch.arange(s["slots"].shape[0], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), token, right=True).clamp(max=held.shape[0] - 1)
    i = token - cu[b]
    at = start[b] + i
    live = token < cu[-1]
    page = s["table"][b, (at // bs).clamp(max=s["table"].shape[1] - 1)].long()
    s["slots"].copy_(torch.where(live, page * bs + at % bs, -1))
    if s["parents"] is not None:
        T = s["parents"].shape[1]
        depth = _ancestors(s["parents"]).sum(-1) - 1
        at = start[b] + torch.where(i < T, depth[b, i.clamp(max=T - 1)], i)
    s["positions"].copy_(torch.where(live, at, 0))
    return [s[x] for x in ("table", "pool", "left", "lens", "cu", "slots", "positions")]


def _own(s):
    from decode_attention_quantized_gb300 import kvq
    op = s["case"]["op"]
    if op == "prompt":
        kvq.kvq_attend_prompt(s["params"], s["q"], s["kn"], s["vn"], s["cu"], s["sink"], s["out"], s["lse"], s["ws"])
        return [s["out"], s["lse"]]
    if op == "tree":
        kvq.kvq_attend_tree(s["cache"], s["params"], s["tree"], s["q"], s["table"], s["lens"], s["sink"], s["out"],
                            s["lse"], s["ws"])
        return [s["out"], s["lse"]]
    if op == "accept":
        kvq.kvq_tree_accept(s["cache"], s["params"], s["tree"], s["drafts"], s["chosen"], s["table"], s["lens"],
                            s["path"], s["accepted"], s["new_lens"], s["next"])
        return _accepted(s)
    kvq.kvq_pages_step(s["params"], s["held"], s["start"], s["new"], s["parents"], s["table"], s["pool"], s["free"],
                       s["lens"], s["left"], s["cu"], s["slots"], s["positions"])
    return [s[x] for x in ("table", "pool", "left", "lens", "cu", "slots", "positions")]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _prompt, "tree": _tree, "accept": _accept, "pages": _pages}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _side64(s, codes, scale, mode, b, h, n):
    """fp64 values of the first n rows of sequence b, kv head h."""
    k, bs = s["k"], s["k"]["block"]
    pages = s["table"][b, :(n + bs - 1) // bs].long()
    c = codes[pages, h].reshape(len(pages) * bs, -1)[:n]
    if k["dtype"] == INT4:
        lo, hi = (c % 16).double(), (c // 16).double()
        v = torch.empty((n, k["d"]), dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = lo - 16 * (lo > 7), hi - 16 * (hi > 7)
    elif k["dtype"] == FP8:
        v = c.view(torch.float8_e4m3fn).double()
    else:
        v = c.double()
        v = v - 256 * (v > 127)
    if mode == ROW:
        return v * scale[pages, h].reshape(-1)[:n, None].double()
    return v * (scale.double() if mode == TENSOR else scale[h].double())


def _rows64(x, vals, cap, hidden, sink):
    """Outputs and log-sum-exps of fp64 scores whose hidden places do not count."""
    if cap > 0:
        x = torch.tanh(x / cap) * cap
    x = x.masked_fill(hidden, -math.inf)
    l = torch.logsumexp(x, -1)
    o = torch.exp(x - l[:, None]) @ vals
    if sink is not None:
        o = o * torch.sigmoid(l - sink.double())[:, None]
    return o, l


def _prompt64(s):
    k, W, at = s["k"], s["case"]["window"], 0
    G = k["hq"] // k["hkv"]
    out, lse = s["out"].double(), s["lse"].double()
    for L in s["lens"]:
        for h in range(k["hq"]):
            keys, vals = (t[at:at + L, h // G].double() for t in (s["kn"], s["vn"]))
            for i0 in range(0, L, 2048):
                i1 = min(L, i0 + 2048)
                j0 = max(0, i0 + 1 - W) if W else 0
                x = s["q"][at + i0:at + i1, h].double() @ keys[j0:i1].T * k["d"] ** -0.5
                far = torch.arange(i0, i1, device="cuda")[:, None] - torch.arange(j0, i1, device="cuda")
                hidden = (far < 0) | (far >= W) if W else far < 0
                o, l = _rows64(x, vals[j0:i1], k["cap"], hidden, None if s["sink"] is None else s["sink"][h])
                out[at + i0:at + i1, h], lse[at + i0:at + i1, h] = o, l
        at += L
    return [out, lse]


def _tree64(s):
    k, case = s["k"], s["case"]
    G, W = k["hq"] // k["hkv"], case["window"]
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    lse = torch.full_like(s["lse"], -math.inf, dtype=torch.float64)
    parents = s["parents"].cpu().numpy()
    for b, (L, n) in enumerate(zip(_lens(case), _nodes(case))):
        P = L - n
        chains = []  # from each node up to its root
        for i in range(n):
            p = int(parents[b, i])
            chains.append([i] + (chains[p] if 0 <= p < i else []))
        hidden = np.ones((n, L), dtype=bool)
        for i, chain in enumerate(chains):
            far = len(chain) - 1  # the node's distance to its root
            hidden[i, (max(0, P + far - W + 1) if W else 0):P] = False
            for up, j in enumerate(chain):
                hidden[i, P + j] = bool(W) and up >= W
        hidden = torch.from_numpy(hidden).cuda()
        for h in range(k["hkv"]):
            keys = _side64(s, s["kc"], s["ks"], k["km"], b, h, L)
            vals = _side64(s, s["vc"], s["vs"], k["vm"], b, h, L)
            for hq in range(h * G, (h + 1) * G):
                x = s["q"][b, :n, hq].double() @ keys.T * k["d"] ** -0.5
                out[b, :n, hq], lse[b, :n, hq] = _rows64(x, vals, k["cap"], hidden,
                                                         None if s["sink"] is None else s["sink"][hq])
    return [out, lse]


def exact(case, seed):
    if case["op"] in ("accept", "pages"):
        return None  # whole numbers, or values moved as they are
    s = prepare(case, seed)
    return _prompt64(s) if case["op"] == "prompt" else _tree64(s)
