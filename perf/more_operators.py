"""The paged cache with rotated keys, measured: appending new tokens to the 16-bit
pages and to the 8-bit pages with the position rotation applied on the way, and
attention of single and drafted tokens over the 16-bit pages.

A 16-bit layer holds K and V in pages of T tokens: [page, token, head, D],
[page, head, token, D], or packed [page, head, token, 2 D] with K first.  An 8-bit
layer holds E4M3 codes and one scale 2^e for each page and head.  The rotation turns
the first R channels of a key or query at position p, in pairs (i, i + R/2) or
(2 i, 2 i + 1), by the angle whose cosine and sine stand in row p of an FP32 table.
``run`` computes each operator in elementary torch operations, or, where ``own`` is
true, makes the calls that a user of ``kv_cache_page_gb300`` makes.
"""
import math
import random

import torch

own = False

E_MIN, E_MAX = -60, 119      # an 8-bit page's scale is 2^e, e within these bounds
CODE_MAX = 448.0             # the largest E4M3 code
THETA = 1e6                  # of the rotation's angles, p * THETA^(-2 i / R)
DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "D": 128, "H": 8, "G": 4, "T": 16, "layout": "nhd", "R": 128,
         "pairs": "halves", "queries": True, "seqs": 1, "idle": 0, "new_lo": 1, "new_hi": 1, "len_lo": 1, "len_hi": 1,
         "causal": True, "window": 0, "shape": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one generated token for each of 64 running sequences, three slots of the batch idle
        _case("append16_step", "append16", seqs=64, idle=3, len_lo=1, len_hi=8192),
        # four whole prompts of 8192 tokens, one layer of the qwen3_8b workload
        _case("append16_prompts", "append16", dtype="fp16", seqs=4, new_lo=8192, new_hi=8192, len_lo=8192, len_hi=8192),
        # prompt chunks of odd lengths in packed pages, a quarter of the channels rotated in neighbouring pairs
        _case("append16_ragged", "append16", D=256, H=2, G=5, T=24, layout="packed", R=64, pairs="neighbours", seqs=23,
              new_lo=0, new_hi=700, len_lo=5, len_hi=1500, shape=2),
        # few users, short contexts: the time to the next token
        _case("step16_small", "attend16", dtype="fp16", seqs=4, len_lo=300, len_hi=600, shape=4),
        # a full batch of uneven contexts, with slots that hold no sequence
        _case("step16_batch", "attend16", seqs=64, idle=3, len_lo=100, len_hi=8192, shape=5),
        # one long context, seven query heads to a KV head
        _case("step16_long", "attend16", H=4, G=7, seqs=1, len_lo=131072, len_hi=131072),
        # one KV head for 32 query heads, packed pages
        _case("step16_one_head", "attend16", dtype="fp16", H=1, G=32, T=64, layout="packed", seqs=48, len_lo=500,
              len_hi=6000, shape=8),
        # drafted tokens checked together, head_dim 256
        _case("step16_draft", "attend16", dtype="fp16", D=256, H=4, G=4, seqs=16, new_lo=2, new_hi=5, len_lo=60,
              len_hi=4096, shape=6),
        # a sliding window over contexts of odd lengths, small pages of an odd size, head_dim 64
        _case("step16_window", "attend16", D=64, H=4, G=2, T=5, layout="hnd", seqs=33, len_lo=1, len_hi=5000, window=1024,
              shape=7),
        # one generated token for each of 64 running sequences, into 8 bits
        _case("append8_step", "append8", dtype="fp16", seqs=64, len_lo=1, len_hi=8192),
        # four whole prompts of 8192 tokens into 8 bits
        _case("append8_prompts", "append8", seqs=4, new_lo=8192, new_hi=8192, len_lo=8192, len_hi=8192),
        # prompt chunks of odd lengths that continue half-filled 8-bit pages, no queries
        _case("append8_ragged", "append8", dtype="fp16", D=64, H=4, T=32, layout="hnd", R=32, queries=False, seqs=23,
              new_lo=0, new_hi=700, len_lo=5, len_hi=1500, shape=2),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["append16", "append16_step", "attend16", "attend16", "attend16", "draft", "append8", "append8_step"])
    op = "attend16" if kind == "draft" else kind.split("_")[0]
    D = rng.choice([32, 64, 128, 128, 256])
    c = _case("", op, dtype=rng.choice(["fp16", "bf16"]), D=D, H=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 5, 7, 8, 16, 32]),
              T=rng.choice([16, 16, 32, 64, 5, 24]), layout=rng.choice(["nhd", "hnd", "packed"] if op != "append8" else ["nhd", "hnd"]),
              R=rng.choice([D, D, D // 2, 16, max(16, 3 * D // 4 // 16 * 16)]), pairs=rng.choice(["halves", "halves", "neighbours"]),
              queries=rng.random() < 0.7, shape=rng.randrange(1 << 30))
    del c["name"]
    wide = c["H"] * D
    if op != "attend16":
        if kind.endswith("_step"):
            c["seqs"], c["len_hi"] = _spread(rng, 1, 256), _spread(rng, 1, 8192)
            c["idle"] = rng.choice([0, 0, 1]) if c["seqs"] > 1 else 0
        else:
            c["seqs"] = _spread(rng, 1, 48)
            # at most as many values as the listed prompts have: 32768 tokens of (2 + 4) x 1024
            most = max(1, min(8192, (6 << 25) // (wide * (2 + (c["G"] if c["queries"] else 0)) * c["seqs"])))
            c["new_hi"] = _spread(rng, 1, most)
            c["new_lo"] = rng.choice([0, 1, c["new_hi"]])
            c["len_hi"] = min(8192, _spread(rng, c["new_hi"], 2 * most))
    else:
        c["window"] = rng.choice([0, 0, 0, 17, 256, 1000])
        c["causal"] = rng.random() < 0.9
        c["seqs"] = _spread(rng, 1, 128)
        c["idle"] = rng.choice([0, 0, 1, c["seqs"] // 3]) if c["seqs"] > 1 else 0
        c["len_hi"] = max(8, _spread(rng, 8, max(64, min(131072, (5 << 25) // (wide * c["seqs"])))))
        if kind == "draft":
            c["new_hi"] = min(rng.choice([2, 3, 4, 8]), c["len_hi"])
            c["new_lo"] = rng.choice([1, c["new_hi"]])
    c["len_lo"] = rng.choice([1, c["len_hi"]])
    return c


def _lengths(case):
    """(tokens held, new ones among them) of each sequence; a property of the case, not of the seed."""
    rng = random.Random(case["shape"])
    lens, new = [], []
    for s in range(case["seqs"]):
        n = rng.randint(case["new_lo"], case["new_hi"]) if s else case["new_hi"]
        lens.append(_spread(rng, max(n, case["len_lo"], 1), max(n, case["len_hi"], 1)))
        new.append(n)
    for s in rng.sample(range(case["seqs"]), case["idle"]):
        lens[s] = 0  # a slot of the batch without a sequence: its rows have no position
    return lens, new


# ------------------------------------------------------------------ inputs
def _page_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX]."""
    m, k = torch.frexp(amax)  # amax = m 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, k - 8, k - 9)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _codes(x, scale):
    """E4M3 codes (bytes) of float32 x against a power of two; beyond the range they saturate."""
    return (x / scale).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _tokens_first(pages, case):
    """[page, token, head, D] of pages in the case's layout."""
    return pages if case["layout"] == "nhd" else pages.transpose(1, 2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    D, H, T, S, dt = case["D"], case["H"], case["T"], case["seqs"], DTYPE[case["dtype"]]
    HQ = H * case["G"]
    lens, new = _lengths(case)
    width = max(1, max(-(-n // T) for n in lens))
    used = sum(-(-n // T) for n in lens)
    pages = used + used // 8 + 2  # some pages are nobody's, the last one among them
    order = torch.randperm(pages - 1, generator=g, device=dev)
    tables = torch.full((S, width), -1, dtype=torch.int32, device=dev)
    places = [s * width + j for s, n in enumerate(lens) for j in range(-(-n // T))]
    tables.view(-1)[torch.tensor(places, dtype=torch.int64, device=dev)] = order[:used].to(torch.int32)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    n_new = cu[-1]
    st = {"case": case, "tables": tables, "lens": lens_d, "n_new": n_new, "max_new": max(new), "max_len": max(lens),
          "cu": None if case["new_lo"] == case["new_hi"] == 1 else torch.tensor(cu, dtype=torch.int32, device=dev)}
    gain = {"k": torch.exp(0.7 * torch.randn(H, D, generator=g, device=dev)), "v": torch.full((H, D), 0.5, device=dev)}

    def values(n, r):
        """K with channels of uneven size and V: the law of the qwen3_8b workload before its rotation."""
        return torch.randn(n, H, D, generator=g, device=dev) * gain[r]

    # which tokens of which pages earlier calls have written
    kept = lens_d.long() if case["op"] == "attend16" else (lens_d.long() - torch.tensor(new, device=dev)).clamp(min=0)
    held = torch.zeros(pages, T, dtype=torch.bool, device=dev)
    flat = tables.view(-1).long()
    left = (kept[:, None] - T * torch.arange(width, device=dev)[None, :]).clamp(0, T).view(-1)
    held[torch.where(flat >= 0, flat, pages - 1)] = (torch.arange(T, device=dev) < left[:, None]) & (flat >= 0)[:, None]
    pools = {}
    for r in "kv":
        if case["op"] == "append8":
            # (smaller than the new tokens' values, so that some pages' scales grow)
            x = torch.where(held[:, :, None, None], 0.25 * values(pages * T, r).view(pages, T, H, D), 0.0)
            scale = torch.exp2(_page_exponent(x.abs().amax(dim=(1, 3))).float())
            x = _codes(x, scale[:, None, :, None])
            st[r + "_scale"] = scale.contiguous()
        else:
            x = values(pages * T, r).view(pages, T, H, D).to(dt)
            if case["op"] == "attend16":  # what no token holds is whatever the memory held, NaN and infinities among it
                noise = torch.randint(-32768, 32768, x.shape, generator=g, device=dev, dtype=torch.int16).view(dt)
                x = torch.where(held[:, :, None, None], x, noise)
        pools[r] = x if case["layout"] == "nhd" else x.transpose(1, 2)
    if case["layout"] == "packed":
        st["packed"] = torch.cat([pools["k"], pools["v"]], dim=3)
        st["k"], st["v"] = st["packed"][..., :D], st["packed"][..., D:]
    else:
        st["k"], st["v"] = pools["k"].contiguous(), pools["v"].contiguous()
    if case["op"] == "attend16":
        st["q"] = torch.randn(n_new, HQ, D, generator=g, device=dev).to(dt)
        st["out"] = torch.empty(n_new, HQ, D, dtype=dt, device=dev)
        st["lse"] = torch.empty(n_new, HQ, dtype=torch.float32, device=dev)
    else:
        # new keys, values and queries side by side, as one projection leaves them
        some = HQ if case["queries"] else 0
        row = torch.empty(n_new, some + 2 * H, D, dtype=dt, device=dev)
        row[:, :some] = torch.randn(n_new, some, D, generator=g, device=dev)
        row[:, some:some + H] = values(n_new, "k")
        row[:, some + H:] = values(n_new, "v")
        st["k_new"], st["v_new"] = row[:, some:some + H], row[:, some + H:]
        if some:
            st["q"], st["q_out"] = row[:, :some], torch.empty(n_new, HQ, D, dtype=dt, device=dev)
        angle = torch.arange(max(1, max(lens)), dtype=torch.float64, device=dev)[:, None] * THETA ** (
            -2.0 * torch.arange(case["R"] // 2, dtype=torch.float64, device=dev) / case["R"])
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    if own:  # what a user's program keeps: the cache's handle, a layer, the step's batch, the rotation, a workspace
        from kv_cache_page_gb300 import cache8, cache16
        strides = {"nhd": (T * H * D, H * D, D), "hnd": (H * T * D, D, T * D), "packed": (2 * H * T * D, 2 * D, 2 * T * D)}
        kw = dict(dtype=case["dtype"], head_dim=D, num_kv_heads=H, num_q_heads=HQ, block_tokens=T, num_blocks=pages,
                  strides=strides[case["layout"]])
        if case["op"] == "append8":
            st["cache"], st["layer"] = cache8.Cache8(**kw), cache8.Layer(st["k"], st["v"], st["k_scale"], st["v_scale"])
        else:
            st["cache"], st["layer"] = cache16.Cache16(**kw), cache16.Layer(st["k"], st["v"])
        st["batch"] = cache8.Batch(st["tables"], st["lens"], st["cu"], n_new=n_new, max_new=st["max_new"],
                                   max_len=st["max_len"])
        if case["op"] == "attend16":
            st["workspace"] = torch.zeros(max(1, st["cache"].attend_workspace(st["batch"])), dtype=torch.uint8, device=dev)
        else:
            st["rotation"] = cache8.Rotation(st["cos"], st["sin"], interleaved=case["pairs"] == "neighbours")
    return st


# ------------------------------------------------------------------ the operators
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        cache, layer, batch = state["cache"], state["layer"], state["batch"]
        if op == "attend16":
            cache.attend(layer, batch, state["q"], state["out"], lse=state["lse"], causal=case["causal"],
                         window=case["window"], workspace=state["workspace"])
        else:
            cache.append(layer, batch, state["k_new"], state["v_new"], rotation=state["rotation"], q=state.get("q"),
                         q_out=state.get("q_out"))
    else:
        {"append16": _plain_append16, "append8": _plain_append8, "attend16": _plain_attend}[op](state)
    if op == "attend16":
        return {"out": state["out"], "lse": state["lse"]}
    result = {"q": state["q_out"]} if "q" in state else {}
    if op == "append8":
        result.update({r: {"codes": state[r].view(torch.float8_e4m3fn), "scale": state[r + "_scale"]} for r in "kv"})
    elif "packed" in state:
        result["pages"] = state["packed"]
    else:
        result.update(k=state["k"], v=state["v"])
    return result


def _starts(state):
    """First row and count of each sequence's new tokens."""
    if state["cu"] is None:
        first = torch.arange(state["lens"].numel(), device=state["lens"].device)
        return first, torch.ones_like(first)
    cu = state["cu"].long()
    return cu[:-1], cu[1:] - cu[:-1]


def _row_places(state):
    """Sequence and position of each new row; a negative position is none."""
    lens, (first, count) = state["lens"].long(), _starts(state)
    row = torch.arange(state["n_new"], device=lens.device)
    seq = torch.searchsorted((first + count).contiguous(), row, right=True)
    return seq, (lens - count - first)[seq] + row


def _rotated(x, pos, state):
    """FP32 values of rows x [n, heads, D] turned by their positions."""
    R, at = state["case"]["R"], pos.clamp(min=0)
    c, s = state["cos"][at][:, None], state["sin"][at][:, None]
    y = x.float()
    halves = state["case"]["pairs"] == "halves"
    a, b = (y[..., :R // 2], y[..., R // 2:R]) if halves else (y[..., 0:R:2], y[..., 1:R:2])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, y[..., R:]], -1)


def _plain_queries(state, pos):
    if "q" in state:
        state["q_out"].copy_(torch.where((pos >= 0)[:, None, None], _rotated(state["q"], pos, state), 0.0))


def _plain_append16(state):
    case, T = state["case"], state["case"]["T"]
    seq, pos = _row_places(state)
    ok, at = pos >= 0, pos.clamp(min=0)
    spare = state["k"].shape[0] - 1  # nobody's page: rows without a position write what its first slot holds
    ids = torch.where(ok, state["tables"].long()[seq, at // T], spare)
    slot = torch.where(ok, at % T, 0)
    for r, x in (("k", _rotated(state["k_new"], pos, state)), ("v", state["v_new"])):
        pool = _tokens_first(state[r], case)
        pool[ids, slot] = torch.where(ok[:, None, None], x.to(pool.dtype), pool[ids, slot])
    _plain_queries(state, pos)


def _plain_append8(state):
    case, T = state["case"], state["case"]["T"]
    lens, (first, count) = state["lens"].long(), _starts(state)
    start = lens - count
    dev = lens.device
    most = (state["max_new"] + T - 2) // T + 1  # pages that a sequence's new tokens touch
    page = (start.clamp(min=0) // T)[:, None] + torch.arange(most, device=dev)[None, :]          # [S, P]
    pos = page[:, :, None] * T + torch.arange(T, device=dev)                                     # [S, P, T]
    is_new = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    before = pos < start[:, None, None]
    touched = is_new.any(2)
    spare = state["k"].shape[0] - 1  # nobody's page, rewritten with what it holds
    ids = torch.where(touched, state["tables"].long().gather(1, page.clamp(max=state["tables"].shape[1] - 1)), spare)
    row = (first[:, None, None] + pos - start[:, None, None]).clamp(0, max(0, state["n_new"] - 1))
    m = is_new[..., None, None]
    fresh = ~(before & touched[..., None]).any(2)[..., None]                                     # nothing to keep
    row_pos = _row_places(state)[1]
    for r, values in (("k", _rotated(state["k_new"], row_pos, state)), ("v", state["v_new"].float())):
        pool, scales = _tokens_first(state[r], case), state[r + "_scale"]
        x = torch.where(m, values[row], 0.0)                                                     # [S, P, T, H, D]
        e = _page_exponent(torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=(2, 4)))
        was = scales[ids]
        scale = torch.exp2(e.float())
        scale = torch.where(fresh, scale, torch.maximum(scale, was))                             # [S, P, H]
        now = scale[:, :, None, :, None]
        old = pool[ids]
        again = _codes(_decode(old) * was[:, :, None, :, None], now)
        got = torch.where(m, _codes(x, now), torch.where(before[..., None, None], again, old))
        pool[ids] = torch.where(touched[..., None, None, None], got, old)
        scales[ids] = torch.where(touched[..., None], scale, was)
    _plain_queries(state, row_pos)


def _plain_attend(state):
    case = state["case"]
    D, H, G, T = case["D"], case["H"], case["G"], case["T"]
    lens, (first, count) = state["lens"].long(), _starts(state)
    S, n, L, dev = lens.numel(), state["max_new"], max(1, state["max_len"]), lens.device
    i = torch.arange(n, device=dev)
    row = (first[:, None] + i).clamp(max=max(0, state["n_new"] - 1))                             # [S, n]
    at = (lens - count)[:, None] + i                                                             # query positions
    j = torch.arange(L, device=dev).expand(S, L)
    held = j < lens[:, None]
    tables = state["tables"].long()
    ids = tables.gather(1, (j // T).clamp(max=tables.shape[1] - 1)).clamp(min=0)
    k, v = (torch.where(held[..., None, None], _tokens_first(state[r], case)[ids, j % T], 0).float() for r in "kv")
    q = state["q"].float()[row].view(S, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(S, H, G, n, L)
    x *= 1.0 / math.sqrt(D)
    see = (held[:, None, :] & (at >= 0)[:, :, None]).expand(S, n, L)
    if case["causal"]:
        see = see & (j[:, None, :] <= at[:, :, None])
    if case["window"]:
        see = see & (j[:, None, :] > at[:, :, None] - case["window"])
    x.masked_fill_(~see[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, H, G * n, L), v.permute(0, 2, 1, 3)).view(S, H, G, n, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = top + torch.log(total)
    # rows beyond a sequence's count land on one spare row
    dst = torch.where(i < count[:, None], first[:, None] + i, state["n_new"]).view(-1)
    out = torch.empty(state["n_new"] + 1, H * G, D, dtype=state["out"].dtype, device=dev)
    out[dst] = o.permute(0, 3, 1, 2, 4).reshape(S * n, H * G, D).to(out.dtype)
    state["out"].copy_(out[:-1])
    back = torch.empty(state["n_new"] + 1, H * G, dtype=torch.float32, device=dev)
    back[dst] = lse.permute(0, 3, 1, 2, 4).reshape(S * n, H * G)
    state["lse"].copy_(back[:-1])


# ------------------------------------------------------------------ what a pass needs
def _seen(case, lens, new):
    """(cached tokens that some row sees, query-key pairs) of a batch."""
    tokens = pairs = 0
    for n, c in zip(lens, new):
        lo, hi = n, 0
        for at in range(max(0, n - c), n):
            a = max(0, at - case["window"] + 1) if case["window"] else 0
            b = at + 1 if case["causal"] else n
            pairs += b - a
            lo, hi = min(lo, a), max(hi, b)
        tokens += max(0, hi - lo)
    return tokens, pairs


def work(case):
    lens, new = _lengths(case)
    D, H, T, R = case["D"], case["H"], case["T"], case["R"]
    HQ, rows = H * case["G"], sum(new)
    if case["op"] == "attend16":
        tokens, pairs = _seen(case, lens, new)
        return {"bytes": 2 * H * tokens * D * 2 + rows * HQ * (2 * 2 * D + 4), "flops": 4 * pairs * HQ * D}
    written = sum(min(n, c) for n, c in zip(lens, new))
    queries = HQ if case["queries"] else 0
    positions, top = 0, 0  # rows of the rotation's table, each once
    for a, b in sorted((max(0, n - c), n) for n, c in zip(lens, new)):
        positions += max(0, b - max(a, top))
        top = max(top, b)
    size = written * H * D * 2 * (2 + (1 if case["op"] == "append8" else 2)) + rows * queries * D * 2 * 2 + positions * R * 4
    if case["op"] == "append8":
        size += 2 * 4 * H * sum(-(-n // T) - (n - c) // T for n, c in zip(lens, new) if c and n)
    return {"bytes": size, "flops": 3 * R * (written * H + rows * queries) + (4 * written * H * D if case["op"] == "append8" else 0)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _e4m3_values(dev):
    """The value of each byte: sign, four exponent bits of bias 7, three mantissa bits; 0x7F and 0xFF are NaN."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    return torch.tensor(out, dtype=torch.float64, device=dev)


def _nearest_e4m3(x):
    """Float64 x to the nearest E4M3 value, ties to even, saturating."""
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _turn(x, start, case, st):
    """Rows x [n, heads, D] in 64 bits, the first at position start, turned as complex numbers."""
    R, n = case["R"], x.shape[0]
    w = torch.complex(st["cos"][start:start + n].double(), st["sin"][start:start + n].double())[:, None]
    y = x.double().clone()
    first = torch.arange(R // 2, device=x.device) * (1 if case["pairs"] == "halves" else 2)
    second = first + (R // 2 if case["pairs"] == "halves" else 1)
    z = torch.complex(y[..., first], y[..., second]) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    lens, new = _lengths(case)
    dev, T, H, D, G = st["lens"].device, case["T"], case["H"], case["D"], case["G"]
    ids = st["tables"].long().cpu()
    if case["op"] == "attend16":
        return _exact_attend(case, st, lens, new, ids)
    result, row = {}, 0
    table = _e4m3_values(dev)
    eight = case["op"] == "append8"
    # [pages, T, H, D] in 64 bits, for 8 bits in units of the scale
    pool = {r: (table[_tokens_first(st[r], case).long()] if eight else _tokens_first(st[r], case).double()).contiguous() for r in "kv"}
    scale = {r: st[r + "_scale"].double() for r in "kv"} if eight else None
    queries = torch.zeros(st["n_new"], H * G, D, dtype=torch.float64, device=dev) if "q" in st else None
    for s, (n, c) in enumerate(zip(lens, new)):
        lost = max(0, c - n)  # rows before the sequence's first token
        if c > lost:
            a, start = (n - c) // T if n >= c else 0, max(0, n - c)
            here, lead, rows = ids[s, a:-(-n // T)].to(dev), max(0, n - c) - a * T, slice(row + lost, row + c)
            if queries is not None:
                queries[rows] = _turn(st["q"][rows], start, case, st)
            for r, x in (("k", _turn(st["k_new"][rows], start, case, st)), ("v", st["v_new"][rows].double())):
                old = pool[r][here].reshape(-1, H, D)
                if not eight:
                    old[lead:lead + c - lost] = x
                    pool[r][here] = old.view(-1, T, H, D)
                    continue
                y = torch.zeros_like(old)
                y[lead:lead + c - lost] = x
                top = y.view(-1, T, H, D).abs().amax(dim=(1, 3))
                want = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(E_MIN, E_MAX))
                want = torch.where(top > 448.0 * want, 2 * want, want)   # where log2 rounded onto a whole number
                want = torch.where((top <= 224.0 * want) & (want > 2.0 ** E_MIN), want / 2, want)
                if lead:
                    was = scale[r][here[0]]
                    want[0] = torch.maximum(want[0], was)
                    y[:lead] = old[:lead] * was[None, :, None]
                y = _nearest_e4m3(y.view(-1, T, H, D) / want[:, None, :, None]).reshape(-1, H, D)
                y[lead + c - lost:] = old[lead + c - lost:]
                pool[r][here], scale[r][here] = y.view(-1, T, H, D), want
        row += c
    if queries is not None:
        result["q"] = queries
    pages = {r: pool[r] if case["layout"] == "nhd" else pool[r].transpose(1, 2).contiguous() for r in "kv"}
    if eight:
        result.update({r: {"codes": pages[r], "scale": scale[r]} for r in "kv"})
    elif case["layout"] == "packed":
        result["pages"] = torch.cat([pages["k"], pages["v"]], dim=3)
    else:
        result.update(pages)
    return result


def _exact_attend(case, st, lens, new, ids):
    T, H, D, G, dev = case["T"], case["H"], case["D"], case["G"], st["lens"].device
    if sum(n * c for n, c in zip(lens, new)) * 4.0 * H * G * D > 8e12:
        return None
    outs, lses, row = [], [], 0
    for s, (n, c) in enumerate(zip(lens, new)):
        if c == 0:
            continue
        q = st["q"][row:row + c].double().view(c, H, G, D)
        row += c
        here = ids[s, :-(-n // T)].to(dev)
        k, v = (_tokens_first(st[r], case)[here].double().reshape(-1, H, D)[:n] for r in "kv")
        o = torch.zeros(c, H, G, D, dtype=torch.float64, device=dev)
        lse = torch.full((c, H, G), -math.inf, dtype=torch.float64, device=dev)
        for i in range(c):
            at = n - c + i
            b = at + 1 if case["causal"] else n
            a = max(0, at - case["window"] + 1) if case["window"] else 0
            if at < 0 or a >= b:
                continue
            z = torch.einsum("hgd,nhd->hgn", q[i], k[a:b]) * D ** -0.5
            lse[i] = torch.logsumexp(z, -1)
            o[i] = torch.einsum("hgn,nhd->hgd", torch.exp(z - lse[i][..., None]), v[a:b])
        outs.append(o.reshape(c, H * G, D))
        lses.append(lse.reshape(c, H * G))
    empty = torch.zeros(0, H * G, D, dtype=torch.float64, device=dev)
    return {"out": torch.cat(outs or [empty]), "lse": torch.cat(lses or [empty[..., 0]])}
