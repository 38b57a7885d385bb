"""Operators over the quantized paged KV cache, as their users call them, and their plain forms.

  attend   attention of a chunk of query tokens (one: a decode step) whose
           scores get a distance bias and an interval of visible keys per token
  mass     the attention weight every cached key received, accumulated
  select   the cache rows that an eviction keeps, by that weight
  compact  the kept rows moved to the front of their sequence's pages

A case is a dict of plain values; sequence lengths, document boundaries and
block counts follow from the case alone, all values from the seed."""
import math
import random

import numpy as np
import torch

own = False

INT8, FP8, INT4 = 1, 2, 3
ROW, TENSOR, CHANNEL = 1, 2, 3
QMAX = {INT8: 127.0, FP8: 448.0, INT4: 7.0}

# cache kinds of the repository's workloads: types, scale modes, heads, block
# size, softcap, and how block ids are laid out
KINDS = {
    "tiny": dict(dtype=INT8, km=ROW, vm=ROW, hq=4, hkv=1, d=64, block=256, cap=0.0),
    "gqa": dict(dtype=INT8, km=ROW, vm=ROW, hq=24, hkv=4, d=256, block=256, cap=0.0),
    "paged": dict(dtype=FP8, km=TENSOR, vm=TENSOR, hq=32, hkv=8, d=128, block=16, cap=50.0),
    "spec": dict(dtype=INT4, km=CHANNEL, vm=CHANNEL, hq=24, hkv=4, d=256, block=32, cap=0.0),
    "mixed": dict(dtype=INT8, km=CHANNEL, vm=TENSOR, hq=64, hkv=8, d=128, block=256, cap=0.0),
}


def listed():
    return [
        # one sequence's decode step inside a short packed document: latency
        dict(name="attend_tiny_document", op="attend", kind="tiny", batch=1, tokens=1, ctx=256, ragged=False,
             bias=False, mask="document"),
        # one long conversation of a model with distance biases, one token a step
        dict(name="attend_decode_bias_long", op="attend", kind="gqa", batch=1, tokens=1, ctx=262144, ragged=False,
             bias=True, mask="causal"),
        # a serving batch of unequal lengths in small shuffled pages
        dict(name="attend_decode_ragged", op="attend", kind="paged", batch=16, tokens=1, ctx=32768, ragged=True,
             bias=True, mask="document"),
        # a prompt of several documents packed into one sequence
        dict(name="attend_prompt_documents", op="attend", kind="gqa", batch=1, tokens=2048, ctx=16384, ragged=False,
             bias=False, mask="document"),
        # prompts of an odd token count whose prefix is seen in both directions
        dict(name="attend_prompt_prefix_odd", op="attend", kind="mixed", batch=3, tokens=509, ctx=8192, ragged=True,
             bias=True, mask="prefix"),
        # the weights of one decode step of a long conversation
        dict(name="mass_decode_long", op="mass", kind="gqa", batch=1, tokens=1, ctx=262144, ragged=False,
             bias=False, mask="causal"),
        # the weights of one decode step of a serving batch
        dict(name="mass_decode_ragged", op="mass", kind="paged", batch=16, tokens=1, ctx=32768, ragged=True,
             bias=False, mask="causal"),
        # the weights that the last 32 tokens of each prompt give to all of it
        dict(name="mass_observe_prompt", op="mass", kind="spec", batch=4, tokens=32, ctx=32768, ragged=False,
             bias=True, mask="causal"),
        # one long conversation cut to a quarter
        dict(name="select_long", op="select", kind="gqa", batch=1, ctx=262144, ragged=False, budget=65536),
        # a large batch of unequal lengths, most of them over the budget
        dict(name="select_ragged", op="select", kind="mixed", batch=64, ctx=131072, ragged=True, budget=4096),
        # one long conversation halved where it lies
        dict(name="compact_long", op="compact", kind="gqa", batch=1, ctx=262144, ragged=False, budget=131072),
        # a serving batch cut to 4096 tokens each, rows of 128 bytes in small pages
        dict(name="compact_ragged", op="compact", kind="paged", batch=16, ctx=32768, ragged=True, budget=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "mass", "mass", "select", "compact"])
    if op == "attend":
        kind = rng.choice(["tiny", "gqa", "paged", "spec", "mixed"])
        if rng.random() < 0.5:
            tokens = rng.choice([1, 1, 2, 5, 8])
            batch = _log(rng, 1, 16)
            ctx = _log(rng, 64, 262144 // batch)
        else:
            tokens = _log(rng, 9, 1500)
            batch = rng.choice([1, 2, 3])
            ctx = tokens + _log(rng, 1, 8192 // batch)
        return dict(op=op, kind=kind, batch=batch, tokens=tokens, ctx=ctx, ragged=rng.random() < 0.5,
                    bias=rng.random() < 0.5, mask=rng.choice(["causal", "document", "prefix"]))
    if op == "mass":
        kind = rng.choice(["tiny", "gqa", "paged", "spec", "mixed"])
        tokens = rng.choice([1, 1, 3, 8, 19, 32, 64])
        batch = _log(rng, 1, 16)
        ctx = tokens + _log(rng, 64, (262144 if tokens <= 8 else 65536) // batch)
        return dict(op=op, kind=kind, batch=batch, tokens=tokens, ctx=ctx, ragged=rng.random() < 0.5,
                    bias=rng.random() < 0.5, mask=rng.choice(["causal", "document"]))
    kind = rng.choice(["tiny", "gqa", "paged", "mixed"])
    if op == "select":
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 256, min(262144, 4194304 // batch))
    else:
        batch = _log(rng, 1, 16)
        ctx = _log(rng, 256, 262144 // batch)
    return dict(op=op, kind=kind, batch=batch, ctx=ctx, ragged=rng.random() < 0.5,
                budget=max(32, _log(rng, ctx // 16, ctx)))


# ------------------------------------------------- what follows from a case

def _lens(case):
    """Sequence lengths: `ctx` for all, or from 1/16 of it to all of it (the
    first sequence has the whole); never shorter than the chunk of queries."""
    r = random.Random("lengths %s" % sorted((k, str(v)) for k, v in case.items() if k != "name"))
    lo = max(case.get("tokens", 1), case["ctx"] // 16, 1)
    if not case["ragged"]:
        return [case["ctx"]] * case["batch"]
    return [case["ctx"]] + [r.randint(lo, max(lo, case["ctx"])) for _ in range(case["batch"] - 1)]


def _intervals(case):
    """key_begin, key_end int32 [B, T] (None: the causal default).  document:
    the token's document begins at the last boundary at or before it; every
    eighth token of a long chunk's end is padding and sees nothing.  prefix:
    the first part of each sequence is seen by every token of it."""
    if case["mask"] == "causal":
        return None, None
    r = random.Random("intervals %s" % sorted((k, str(v)) for k, v in case.items() if k != "name"))
    B, T = case["batch"], case["tokens"]
    begin, end = np.zeros((B, T), np.int32), np.zeros((B, T), np.int32)
    for b, L in enumerate(_lens(case)):
        pos = L - T + np.arange(T)
        end[b] = pos + 1
        if case["mask"] == "document":
            cuts = [0]
            while cuts[-1] < L:
                cuts.append(cuts[-1] + max(1, _log(r, max(1, L // 32), max(2, L // 2))))
            cuts = np.array(cuts)
            begin[b] = cuts[np.searchsorted(cuts, pos, side="right") - 1]
            if T >= 64:
                end[b, -(T // 64):] = 0
        else:
            end[b] = np.maximum(end[b], r.randint(L // 4, L))
    return (begin if case["mask"] == "document" else None), end


def _visible(case):
    """Per sequence: keys that some token sees, and visible (token, key) pairs."""
    begin, end = _intervals(case)
    T, got = case["tokens"], []
    for b, L in enumerate(_lens(case)):
        pos = L - T + np.arange(T)
        lo = np.zeros(T, np.int64) if begin is None else begin[b].astype(np.int64)
        hi = pos + 1 if end is None else end[b].astype(np.int64)
        n = np.maximum(0, hi - lo)
        mark = np.zeros(L + 1, np.int64)
        np.add.at(mark, lo[n > 0], 1)
        np.add.at(mark, hi[n > 0], -1)
        got.append((int((np.cumsum(mark)[:L] > 0).sum()), int(n.sum())))
    return got


def _row_bytes(k, side=None):
    """Bytes of one cached row (a side's codes and its row scale)."""
    code = k["d"] // 2 if k["dtype"] == INT4 else k["d"]
    sides = {"k": [k["km"]], "v": [k["vm"]], None: [k["km"], k["vm"]]}[side]
    return sum(code + (4 if m == ROW else 0) for m in sides)


def work(case):
    k, lens = KINDS[case["kind"]], _lens(case)
    tables = 4 * sum((L + k["block"] - 1) // k["block"] for L in lens) + 4 * len(lens)
    if case["op"] in ("attend", "mass"):
        rows = case["batch"] * case["tokens"] * k["hq"]
        seen = _visible(case)
        pairs = sum(p for _, p in seen) * k["hq"]
        masks = 0 if case["mask"] == "causal" else 8 * case["batch"] * case["tokens"]
        if case["op"] == "attend":
            return dict(bytes=sum(n for n, _ in seen) * k["hkv"] * _row_bytes(k) + rows * (4 * k["d"] + 4) + tables + masks,
                        flops=4 * k["d"] * pairs)
        return dict(bytes=sum(n for n, _ in seen) * k["hkv"] * _row_bytes(k, "k") + rows * (2 * k["d"] + 4)
                    + 8 * sum(lens) * k["hkv"] + tables + masks, flops=2 * k["d"] * pairs)
    kept = sum(min(L, case["budget"]) for L in lens) * k["hkv"]
    if case["op"] == "select":
        return dict(bytes=4 * sum(lens) * k["hkv"] + 4 * kept + tables, flops=0)
    return dict(bytes=kept * (2 * (_row_bytes(k) + 4) + 4) + tables, flops=0)


# ------------------------------------------------------------------ inputs

def _bias_slopes(hq):
    """The usual geometric ladder of distance slopes, 2^(-8 (h + 1) / Hq)."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device="cuda")


def _make_side(k, mode, blocks, g, spread):
    """Codes and scales of one side, drawn in the cache's own layout
    [blocks, Hkv, block, D]: normal values (K channels of unequal size),
    quantized as the cache holds them."""
    hkv, bs, d, dt = k["hkv"], k["block"], k["d"], k["dtype"]
    f = torch.exp(spread * torch.randn((hkv, 1, d), generator=g, device="cuda"))
    per_row = mode == ROW
    scale = torch.empty((blocks, hkv, bs), dtype=torch.float32, device="cuda") if per_row else None
    codes = torch.empty((blocks, hkv, bs, d // 2 if dt == INT4 else d), dtype=torch.uint8, device="cuda")
    if mode == TENSOR:
        scale = torch.full((1,), 5.0 / QMAX[dt], device="cuda")
    if mode == CHANNEL:
        scale = (f[:, 0] * 4.5 / QMAX[dt]).contiguous()
    step = max(1, (1 << 27) // (hkv * bs * d))
    for i in range(0, blocks, step):
        x = torch.randn((min(step, blocks - i), hkv, bs, d), generator=g, device="cuda") * f
        if per_row:
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


def prepare(case, seed):
    k, lens = KINDS[case["kind"]], _lens(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, bs, top = case["batch"], k["block"], max(lens)
    need = [(L + bs - 1) // bs for L in lens]
    blocks, width = sum(need), max(need)
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    if k["block"] == 256:
        perm = torch.arange(blocks, dtype=torch.int32, device="cuda")
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    s = dict(case=case, k=k, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), top=top)
    # weights that some eight decayed steps of a kv head's query heads have left
    s["mass"] = torch.empty((blocks, k["hkv"], bs), device="cuda").exponential_(1.0, generator=g)
    s["mass"] *= 8.0 * k["hq"] / k["hkv"] / top
    op = case["op"]
    if op != "select":
        s["kc"], s["ks"] = _make_side(k, k["km"], blocks, g, 0.5)
        if op != "mass":
            s["vc"], s["vs"] = _make_side(k, k["vm"], blocks, g, 0.0)
        else:
            s["vc"], s["vs"] = s["kc"], s["ks"]  # the weights need no values
    if op in ("attend", "mass"):
        T = case["tokens"]
        s["q"] = torch.randn((B, T, k["hq"], k["d"]), generator=g, device="cuda").to(torch.bfloat16)
        s["slopes"] = _bias_slopes(k["hq"]) if case["bias"] else None
        begin, end = _intervals(case)
        s["begin"] = None if begin is None else torch.from_numpy(begin).cuda()
        s["end"] = None if end is None else torch.from_numpy(end).cuda()
        s["sink"] = torch.randn((k["hq"],), generator=g, device="cuda") if case["kind"] == "mixed" and op == "attend" else None
        s["out"] = torch.empty((B, T, k["hq"], k["d"]), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, T, k["hq"]), dtype=torch.float32, device="cuda")
        if op == "mass":
            s["lse"].copy_(_lse_of(_scores(s)).to(torch.float32))
    else:
        s["sinks"], s["recent"] = min(4, case["budget"] // 8), case["budget"] // 8
        s["keep"] = torch.full((B, k["hkv"], case["budget"]), -1, dtype=torch.int32, device="cuda")
        s["kept"] = torch.clamp(s["lens"], max=case["budget"])
        if op == "compact":
            # what a selection gives: ascending rows, sinks and the newest among them
            for b, L in enumerate(lens):
                n = min(L, case["budget"])
                order = torch.rand((k["hkv"], L), generator=g, device="cuda")
                order[:, :s["sinks"]] = -1.0
                order[:, L - s["recent"]:] = -1.0
                s["keep"][b, :, :n] = order.topk(n, dim=1, largest=False).indices.sort(dim=1).values.to(torch.int32)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors, workspace and plan that a user's program keeps."""
    from decode_attention_quantized_gb300 import kvq
    case, k = s["case"], s["k"]
    blocks, (B, width) = s["mass"].shape[0], s["table"].shape
    if case["op"] != "select":
        one = torch.ones((1,), device="cuda")
        c = s["cache"] = kvq.QuantizedPagedCache(k["dtype"], kvq.PER_TENSOR, kvq.PER_TENSOR, 1, k["block"], k["hkv"],
                                                 k["d"], k_static=one, v_static=one)
        c.num_blocks, c.k_mode, c.v_mode = blocks, k["km"], k["vm"] if case["op"] != "mass" else k["km"]
        c.k_codes, c.v_codes, c.k_scale, c.v_scale = s["kc"], s["vc"], s["ks"], s["vs"]
    n = 0
    if case["op"] in ("attend", "mass"):
        s["params"] = kvq.make_params(B, k["hq"], case["tokens"], width, max_seq_len=s["top"], softcap=k["cap"])
        s["mask"] = kvq.ScoreMask(slopes=s["slopes"], key_begin=s["begin"], key_end=s["end"])
        size = (kvq.kvq_attend_masked_workspace_size if case["op"] == "attend" else kvq.kvq_key_mass_workspace_size)
        n = size(s["cache"], s["params"])
    else:
        s["eparams"] = kvq.make_evict_params(B, width, case["budget"], num_blocks=blocks, block_size=k["block"],
                                             num_kv_heads=k["hkv"], sinks=s["sinks"], recent=s["recent"],
                                             max_seq_len=s["top"])
        if case["op"] == "compact":
            n = kvq.kvq_evict_compact_workspace_size(s["cache"], s["eparams"])
    s["ws"] = torch.empty(n // 4 + 64, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- plain forms

def _rows(s):
    """Block and row of every position [B, 1, top], and which positions exist."""
    at = torch.arange(s["top"], device="cuda")
    return (s["table"][:, at // s["k"]["block"]].long()[:, None], (at % s["k"]["block"])[None, None],
            at[None] < s["lens"][:, None])


def _values(s, codes, scale, mode):
    """The fp32 values of a side's rows in sequence order, [B, Hkv, top, D]."""
    k = s["k"]
    blk, row, _ = _rows(s)
    head = torch.arange(k["hkv"], device="cuda")[None, :, None]
    c = codes[blk, head, row]
    if k["dtype"] == INT4:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
        c = torch.where(c >= 8, c - 16, c)
    else:
        c = c.view(torch.int8 if k["dtype"] == INT8 else torch.float8_e4m3fn).float()
    if mode == ROW:
        return c * scale[blk, head, row][..., None]
    return c * (scale if mode == TENSOR else scale[:, None, :])


def _scores(s):
    """fp32 scores [B, Hkv, T, G, top], -inf where a row does not see a key."""
    k, T = s["k"], s["case"]["tokens"]
    B, G, top = s["q"].shape[0], k["hq"] // k["hkv"], s["top"]
    q = s["q"].float().reshape(B, T, k["hkv"], G, k["d"]).transpose(1, 2).reshape(B, k["hkv"], T * G, k["d"])
    x = q @ _values(s, s["kc"], s["ks"], k["km"]).transpose(2, 3) / math.sqrt(k["d"])
    if k["cap"] > 0:
        x = k["cap"] * torch.tanh(x / k["cap"])
    x = x.reshape(B, k["hkv"], T, G, top)
    key = torch.arange(top, device="cuda")
    pos = s["lens"][:, None] - T + torch.arange(T, device="cuda")
    if s["slopes"] is not None:
        far = (pos[:, :, None] - key).abs().float()
        x = x - s["slopes"].reshape(1, k["hkv"], 1, G, 1) * far[:, None, :, None]
    end = pos + 1 if s["end"] is None else s["end"]
    end = torch.minimum(end, s["lens"][:, None])
    see = key < end[:, :, None]
    if s["begin"] is not None:
        see = see & (key >= s["begin"][:, :, None])
    return torch.where(see[:, None, :, None], x, -math.inf)


def _lse_of(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    return (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True)))[..., 0].permute(0, 2, 1, 3).flatten(2)


def _attend(s):
    k, T = s["k"], s["case"]["tokens"]
    x = _scores(s)
    B, hkv, _, G, top = x.shape
    lse = _lse_of(x)
    by_head = lse.reshape(B, T, hkv, G).permute(0, 2, 1, 3)[..., None]
    p = torch.exp(x - torch.where(by_head == -math.inf, 0.0, by_head))
    live = _rows(s)[2][:, None, :, None]
    v = torch.where(live, _values(s, s["vc"], s["vs"], k["vm"]), 0.0)
    o = (p.reshape(B, hkv, T * G, top) @ v).reshape(B, hkv, T, G, k["d"])
    if s["sink"] is not None:
        o = o / (1.0 + torch.exp(s["sink"].reshape(1, hkv, 1, G, 1) - by_head))
        o = torch.where(by_head == -math.inf, 0.0, o)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(s["out"].shape))
    s["lse"].copy_(lse)
    return [s["out"], s["lse"]]


DECAY = 0.875


def _mass(s):
    k, T = s["k"], s["case"]["tokens"]
    x = _scores(s)
    B, hkv, _, G, top = x.shape
    by_head = s["lse"].reshape(B, T, hkv, G).permute(0, 2, 1, 3)[..., None]
    p = torch.exp(x - torch.where(by_head == -math.inf, 0.0, by_head)).sum((2, 3))
    blk, row, live = _rows(s)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    old = s["mass"][blk, head, row]
    fresh = torch.arange(top, device="cuda")[None] >= s["lens"][:, None] - T
    new = p + torch.where(fresh[:, None], 0.0, DECAY * old)
    live = live[:, None].expand(B, hkv, top)
    s["mass"][blk.expand(B, hkv, top)[live], head.expand(B, hkv, top)[live], row.expand(B, hkv, top)[live]] = new[live]
    return s["mass"]


def _select(s):
    k, n = s["k"], s["case"]["budget"]
    blk, row, live = _rows(s)
    head = torch.arange(k["hkv"], device="cuda")[None, :, None]
    m = s["mass"][blk, head, row]
    at, lens = torch.arange(s["top"], device="cuda")[None], s["lens"][:, None]
    sure = (at < s["sinks"]) | (at >= lens - s["recent"])
    m = torch.where(sure[:, None], math.inf, m)
    m = torch.where(live[:, None], m, -math.inf)
    order = torch.sort(m, dim=-1, descending=True, stable=True).indices[..., :n]
    chosen = torch.zeros(m.shape, dtype=torch.bool, device="cuda").scatter_(-1, order, True) & live[:, None]
    rank = torch.cumsum(chosen, -1) - 1
    s["keep"].fill_(-1)
    b, h, i = chosen.nonzero(as_tuple=True)
    s["keep"][b, h, rank[b, h, i]] = i.to(torch.int32)
    s["kept"].copy_(torch.clamp(s["lens"], max=n))
    return [s["keep"], s["kept"]]


def _compact(s):
    k, bs = s["k"], s["k"]["block"]
    b, h, i = (s["keep"] >= 0).nonzero(as_tuple=True)
    src = s["keep"][b, h, i].long()
    sb, sr = s["table"][b, src // bs].long(), src % bs
    db, dr = s["table"][b, i // bs].long(), i % bs
    s["kc"][db, h, dr] = s["kc"][sb, h, sr]
    s["vc"][db, h, dr] = s["vc"][sb, h, sr]
    if k["km"] == ROW:
        s["ks"][db, h, dr] = s["ks"][sb, h, sr]
    if k["vm"] == ROW:
        s["vs"][db, h, dr] = s["vs"][sb, h, sr]
    s["mass"][db, h, dr] = s["mass"][sb, h, sr]
    return _compacted(s)


def _compacted(s):
    kind = torch.int8 if s["k"]["dtype"] == INT8 else torch.float8_e4m3fn
    return [s["kc"].view(kind), s["vc"].view(kind), s["ks"], s["vs"], s["mass"]]


def _own(s):
    from decode_attention_quantized_gb300 import kvq
    op = s["case"]["op"]
    if op == "attend":
        kvq.kvq_attend_masked(s["cache"], s["params"], s["mask"], s["q"], s["table"], s["lens"], s["sink"], s["out"],
                              s["lse"], s["ws"])
        return [s["out"], s["lse"]]
    if op == "mass":
        kvq.kvq_key_mass(s["cache"], s["params"], s["mask"], s["q"], s["table"], s["lens"], s["lse"], s["mass"],
                         s["ws"], decay=DECAY)
        return s["mass"]
    if op == "select":
        kvq.kvq_evict_select(s["eparams"], s["mass"], s["table"], s["lens"], s["keep"], s["kept"])
        return [s["keep"], s["kept"]]
    kvq.kvq_evict_compact(s["cache"], s["eparams"], s["table"], s["table"], s["keep"], s["kept"], s["mass"], s["ws"])
    return _compacted(s)


def run(state):
    if own:
        return _own(state)
    return {"attend": _attend, "mass": _mass, "select": _select, "compact": _compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _side64(s, codes, scale, mode, b, h, n):
    """fp64 values of the first n rows of sequence b, kv head h."""
    k = s["k"]
    bs = k["block"]
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


def _scores64(s, b, hq, keys):
    """fp64 scores [T, n] of query head hq of sequence b against its keys."""
    k, T, n = s["k"], s["case"]["tokens"], keys.shape[0]
    x = (s["q"][b, :, hq].double() @ keys.T) * k["d"] ** -0.5
    if k["cap"] > 0:
        x = torch.tanh(x / k["cap"]) * k["cap"]
    for t0 in range(0, T, 256):
        t1 = min(T, t0 + 256)
        pos = torch.arange(n - T + t0, n - T + t1, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        if s["slopes"] is not None:
            x[t0:t1] -= s["slopes"][hq].double() * (pos - j).abs()
        hidden = j > pos if s["end"] is None else j >= s["end"][b, t0:t1, None]
        if s["begin"] is not None:
            hidden = hidden | (j < s["begin"][b, t0:t1, None])
        x[t0:t1].masked_fill_(hidden, -math.inf)
    return x


def exact(case, seed):
    op, k = case["op"], KINDS[case["kind"]]
    if op in ("select", "compact"):
        return None  # whole numbers, or values moved as they are
    s = prepare(case, seed)
    G = k["hq"] // k["hkv"]
    lens = _lens(case)
    if op == "attend":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        mass = s["mass"].double()
    for b, n in enumerate(lens):
        for h in range(k["hkv"]):
            keys = _side64(s, s["kc"], s["ks"], k["km"], b, h, n)
            if op == "attend":
                vals = _side64(s, s["vc"], s["vs"], k["vm"], b, h, n)
            else:
                got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for hq in range(h * G, (h + 1) * G):
                x = _scores64(s, b, hq, keys)
                if op == "mass":
                    l = s["lse"][b, :, hq, None].double()
                    got += torch.exp(x - torch.where(torch.isfinite(l), l, 0.0)).sum(0)
                    continue
                l = torch.logsumexp(x, 1)
                lse[b, :, hq] = l
                o = torch.exp(x - torch.where(torch.isfinite(l), l, 0.0)[:, None]) @ vals
                if s["sink"] is not None:
                    o = o * torch.sigmoid(l - s["sink"][hq].double())[:, None]
                out[b, :, hq] = o
            if op == "mass":
                pages = s["table"][b, :(n + k["block"] - 1) // k["block"]].long()
                rows = mass[pages, h].reshape(-1)
                rows[:n] = got + torch.cat([rows[:n - case["tokens"]] * DECAY, torch.zeros_like(got[:case["tokens"]])])
                mass[pages, h] = rows.reshape(len(pages), -1)
    return [out, lse] if op == "attend" else mass
