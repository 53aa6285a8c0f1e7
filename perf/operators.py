"""The dense side of a paged KV cache, measured: page allocation with the slot map of a
batch's new tokens, the write of those tokens' rows, and the attention of one new token over
the whole cache.

Three operators, in the order a serving step uses them:

* ``tables``  se_block_tables_extend and se_block_tables_release: pages for every request's
  new tokens from a pool of free pages, the block-table entries, the slot and the position of
  every new token; then the pages back to the pool.
* ``store``   se_paged_kv_store: the K and V rows of a ragged batch of new tokens into their
  slots, with the pages' key minima and maxima where the cache keeps them.
* ``decode``  se_paged_decode: softmax(sm_scale q k) v of one query token per request over its
  cached tokens, all of them or the first ``sink`` and the last ``recent``.

``own`` chooses between the plain form (torch operations in fp32) and the library's calls.
"""
import math

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of 32 requests at 64K-128K tokens: one token each, a page now and then.
        _tables("tables_decode_b32", batch=32, before=(65536, 131072), new=(1, 1)),
        # Four 32K-token prompts admitted at once: 8,192 pages, 131,072 slots.
        _tables("tables_prefill_b4_32k", batch=4, before=(0, 0), new=(32768, 32768)),
        # Chunked prefill beside decoding requests: 250 requests with 1 to 2,500 new tokens each.
        _tables("tables_mixed_b250", batch=250, before=(0, 20011), new=(1, 2500)),
        # The rows of one decode step of 32 requests (4 KV heads), with the page summaries.
        _store("store_decode_b32", batch=32, inside=True, new=(1, 1), heads=4, q_heads=32, dim=128),
        # Four 32K-token prompts, 8 KV heads, read out of the fused QKV projection's output.
        _store("store_prefill_b4_32k", batch=4, inside=False, new=(32768, 32768), heads=8, q_heads=32, dim=128),
        # Prompt chunks of odd lengths for a latent cache: one 576-wide row per token.
        _store("store_latent_b9", batch=9, inside=True, new=(1, 15001), heads=1, q_heads=0, dim=576),
        # The smallest decode: one request, 4,096 tokens, one KV head.
        _decode("decode_b1_g4_4k", batch=1, lens=(4096, 4096), q_heads=4, heads=1, dim=128),
        # The compacted caches that an eviction leaves: 2,048 kept tokens and those decoded since.
        _decode("decode_compacted_b4_2k", batch=4, lens=(2048, 3040), q_heads=32, heads=8, dim=128),
        # 32K contexts, 8 KV heads.
        _decode("decode_b8_32k", batch=8, lens=(32768, 32768), q_heads=32, heads=8, dim=128),
        # Sink and recent windows over ragged histories, some requests still empty.
        _decode("decode_window_b48", batch=48, lens=(0, 33001), q_heads=32, heads=4, dim=128, sink=64, recent=1000),
        # A latent cache at 32K: 64 heads share one row per token.
        _decode("decode_latent_b64_32k", batch=64, lens=(32768, 32768), q_heads=64, heads=1, dim=576),
        # The headline shape's dense layers: ragged 64K-128K contexts, 32 requests.
        _decode("decode_b32_128k", batch=32, lens=(65536, 131072), q_heads=32, heads=4, dim=128),
    ]


def _tables(name, batch, before, new):
    return {"name": name, "op": "tables", "batch": batch, "before_min": before[0], "before_max": before[1],
            "new_min": new[0], "new_max": new[1]}


def _store(name, batch, inside, new, heads, q_heads, dim, summary=True):
    """``inside``: requests already hold tokens, so that their first new one may land inside a page."""
    return {"name": name, "op": "store", "batch": batch, "inside": inside, "new_min": new[0], "new_max": new[1],
            "kv_heads": heads, "q_heads": q_heads, "dim": dim, "summary": summary}


def _decode(name, batch, lens, q_heads, heads, dim, sink=0, recent=0):
    return {"name": name, "op": "decode", "batch": batch, "len_min": lens[0], "len_max": lens[1], "q_heads": q_heads,
            "kv_heads": heads, "dim": dim, "sink": sink, "recent": recent}


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "decode", "decode"])
    if op == "tables":
        batch = _log(rng, 1, 512)
        new = _log(rng, 1, max(1, min(32768, 600000 // batch)))
        before = rng.choice([0, _log(rng, 1, 131072)])
        c = _tables("", batch, (before // 2, before), (rng.choice([0, 1, new]), new))
    elif op == "store":
        heads, q_heads, dim = rng.choice([(1, 4, 128), (2, 12, 128), (4, 32, 128), (8, 32, 128), (3, 9, 128),
                                          (8, 0, 64), (4, 16, 256), (1, 0, 576)])
        batch = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, min(32768, (131072 * 8 // max(heads, 4)) // batch)))
        c = _store("", batch, rng.random() < 0.7, (rng.choice([1, new]), new), heads, q_heads, dim,
                   summary=rng.random() < 0.7)
    else:
        # Query and KV heads: groups of 1 to 64, KV head counts that are no power of two among them.
        q_heads, heads, dim = rng.choice([(4, 1, 128), (8, 8, 128), (16, 2, 128), (32, 8, 128), (32, 4, 128),
                                          (28, 4, 128), (40, 8, 128), (10, 10, 128), (9, 3, 128), (32, 1, 128),
                                          (64, 8, 64), (12, 4, 64), (16, 8, 256), (8, 1, 256),
                                          (16, 1, 576), (32, 1, 576), (48, 1, 576), (64, 1, 576)])
        longest = _log(rng, 1, 131072)
        row = heads * dim * (2 if dim == 576 else 4)
        batch = _log(rng, 1, max(1, min(256, 3_200_000_000 // (row * longest))))
        sink, recent = (0, 0) if rng.random() < 0.6 else (rng.choice([0, 4, 64, _log(rng, 1, 500)]), _log(rng, 1, 4096))
        c = _decode("", batch, (rng.choice([0, 1, longest // 2, longest]), longest), q_heads, heads, dim, sink, recent)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _lengths(lo, hi, batch, g):
    return torch.randint(lo, hi + 1, (batch,), generator=g)


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _normal(shape, g):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _paged(tokens, perm, width):
    """Block table [batch][width] of requests of these lengths over the pages of ``perm``, in order; unused
    entries 0."""
    n = _pages(tokens)
    at = torch.cumsum(n, 0) - n
    p = torch.arange(width)
    idx = at[:, None] + p[None]
    inside = p[None] < n[:, None]
    return torch.where(inside, perm[torch.where(inside, idx, torch.zeros_like(idx))], torch.zeros_like(idx)).int()


def _host_slots(before, new, table):
    """Slots of the new tokens, request after request (on the host)."""
    batch = before.numel()
    r = torch.repeat_interleave(torch.arange(batch), new)
    pos = before[r] + torch.arange(r.numel()) - (torch.cumsum(new, 0) - new)[r]
    return table[r, pos // PAGE] * PAGE + (pos % PAGE).int()


def prepare(case, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    dg = torch.Generator("cuda").manual_seed(seed)
    state = {"case": case}
    batch = case["batch"]
    if case["op"] == "decode":
        lens = _lengths(case["len_min"], case["len_max"], batch, g)
        total = max(1, int(_pages(lens).sum()))
        perm = torch.randperm(total, generator=g)
        width = max(1, int(_pages(lens).max()))
        state["block_table"] = _paged(lens, perm, width).cuda()
        state["seq_lens"] = lens.int().cuda()
        hq, h, d = case["q_heads"], case["kv_heads"], case["dim"]
        state["dv"] = dv = 512 if d == 576 else d
        state["sm_scale"] = 1.0 / math.sqrt(d)
        k = _normal((total, h, PAGE, d), dg)
        # A few key channels per head are larger than the others, as in real caches.
        scale = torch.ones(h, 1, d, dtype=torch.bfloat16)
        for i in range(h):
            scale[i, 0, torch.randperm(d, generator=g)[:4]] = 4.0
        k.mul_(scale.cuda())
        v = None if d == 576 else _normal((total, h, PAGE, dv), dg)
        # What lies behind a request's last token in its last page is stale: NaN here.
        last = (lens - 1).clamp_min(0) // PAGE
        phys = state["block_table"].cpu().long()[torch.arange(batch), last]
        slot = torch.arange(PAGE)
        stale = (slot[None] >= (lens - last * PAGE)[:, None]) & (lens > 0)[:, None]
        pi, si = (x.cuda() for x in (phys[:, None].expand(-1, PAGE)[stale], slot[None].expand(batch, -1)[stale]))
        k[pi, :, si] = float("nan")
        if v is not None:
            v[pi, :, si] = float("nan")
        state.update(k=k, v=v, q=_normal((batch, hq, d), dg))
        state["out"] = torch.empty(batch, hq, dv, dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.empty(batch, hq, dtype=torch.float32, device="cuda")
        if own:  # the cache view and the workspace that a program keeps
            import sparse_decode_attention_quest_gb300 as se
            state["kv"] = se.paged_kv(k, v, None, dv)
            ws = se.se_paged_decode_workspace_size(batch, hq, h, d, dv)
            state["workspace"] = torch.zeros(ws, dtype=torch.uint8, device="cuda")
        return state
    new = _lengths(case["new_min"], case["new_max"], batch, g)
    if case["op"] == "tables":
        before = _lengths(case["before_min"], case["before_max"], batch, g)
        width = _pages(case["before_max"] + case["new_max"])
        num_pages = batch * width + 16
        perm = torch.randperm(num_pages, generator=g)
        held = int(_pages(before).sum())
        state["block_table"] = _paged(before, perm, width).cuda()
        # The free pages: a stack, taken from its end; the rest of the array is unused.
        free = torch.zeros(num_pages, dtype=torch.int32)
        free[: num_pages - held] = perm[held:].int()
        state["free_pages"] = free.cuda()
        state["pool_state"] = torch.tensor([num_pages - held, 0, 0, 0], dtype=torch.int32, device="cuda")
        state["before"], state["new"] = before.int().cuda(), new.int().cuda()
        # The slot map is as long as the largest batch of tokens that the program takes.
        longest = max(1, batch * case["new_max"])
        state["after"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        state["token_start"] = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
        state["slot_map"] = torch.zeros(longest, dtype=torch.int32, device="cuda")
        state["positions"] = torch.zeros(longest, dtype=torch.int32, device="cuda")
        return state
    # The pool holds the pages that take new tokens, in any order.
    inside = _lengths(0, PAGE - 1, batch, g) if case["inside"] else torch.zeros_like(new)
    tokens = int(new.sum())
    width = _pages((PAGE - 1 if case["inside"] else 0) + case["new_max"])
    pages = batch * width
    table = _paged(inside + new, torch.randperm(pages, generator=g), width)
    state["slot_map"] = _host_slots(inside, new, table).int().cuda()
    h, hq, d = case["kv_heads"], case["q_heads"], case["dim"]
    state["k"] = _normal((pages, h, PAGE, d), dg)
    state["v"] = None if d == 576 else _normal((pages, h, PAGE, d), dg)
    # Key and value rows: columns of the fused projection's output (the queries before them).
    fused = _normal((tokens, hq + (1 if d == 576 else 2) * h, d), dg)
    state["k_new"] = fused[:, hq:hq + h]
    state["v_new"] = None if d == 576 else fused[:, hq + h:]
    state["summary"] = None
    if case["summary"]:
        mid = _normal((pages, h, 1, d), dg)
        half = _normal((pages, h, 1, d), dg).abs_()
        state["summary"] = torch.cat([mid - half, mid + half], 2).contiguous()
    if own:
        import sparse_decode_attention_quest_gb300 as se
        state["kv"] = se.paged_kv(state["k"], state["v"], state["summary"], 512 if d == 576 else d)
    return state


# ------------------------------------------------------------------ plain forms
def _tables_plain(s):
    before, new = s["before"].long(), s["new"].long()
    table, free, slot_map = s["block_table"], s["free_pages"], s["slot_map"]
    start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    have, after = _pages(before), before + new
    need = _pages(after) - have
    off = torch.cumsum(need, 0) - need
    count = s["pool_state"][0].long()
    # Page p of request b, opened by this call: the free page off_b + p - have_b from the stack's end.
    p = torch.arange(table.shape[1], device="cuda")[None]
    opened = (p >= have[:, None]) & (p < (have + need)[:, None])
    at = torch.where(opened, count - 1 - (off[:, None] + p - have[:, None]), torch.zeros_like(p))
    table.copy_(torch.where(opened, free[at], table))
    t = torch.arange(slot_map.numel(), device="cuda")
    inside = t < start[-1]
    r = torch.searchsorted(start[1:], t, right=True).clamp_max(new.numel() - 1)
    pos = torch.where(inside, before[r] + t - start[r], torch.zeros_like(t))
    slot_map.copy_(torch.where(inside, table[r, pos // PAGE].long() * PAGE + pos % PAGE, torch.full_like(t, -1)))
    s["positions"].copy_(pos)
    s["after"].copy_(after)
    s["token_start"].copy_(start)
    s["pool_state"][0] = count - need.sum()
    # ... and back: the pages behind ceil(before / 16) of every request onto the stack.
    back = _pages(s["after"].long()) - have
    off = torch.cumsum(back, 0) - back
    total = s["pool_state"][0].long() + back.sum()
    mine = (p >= have[:, None]) & (p < (have + back)[:, None])
    to = torch.where(mine, total - 1 - (off[:, None] + p - have[:, None]), torch.full_like(p, free.numel()))
    room = torch.cat([free, free[:1]])
    room.scatter_(0, to.reshape(-1), table.reshape(-1))
    free.copy_(room[:-1])
    s["pool_state"][0] = total
    return _tables_out(s)


def _tables_out(s):
    return {k: s[k] for k in ("block_table", "slot_map", "positions", "after", "token_start", "free_pages",
                              "pool_state")}


def _store_plain(s):
    slot = s["slot_map"].long()
    page, off = slot // PAGE, slot % PAGE
    s["k"][page, :, off] = s["k_new"]
    if s["v"] is not None:
        s["v"][page, :, off] = s["v_new"]
    if s["summary"] is not None:
        pages, h, _, d = s["k"].shape
        # Pages whose first token is among the new ones start anew, the others take theirs in.
        fresh = torch.zeros(pages, dtype=torch.int32, device="cuda").scatter_reduce(0, page, (off == 0).int(), "amax") > 0
        inf = torch.full((), math.inf, device="cuda")
        lo = torch.where(fresh[:, None, None], inf, s["summary"][:, :, 0].float())
        hi = torch.where(fresh[:, None, None], -inf, s["summary"][:, :, 1].float())
        idx = page[:, None, None].expand(-1, h, d)
        lo = lo.scatter_reduce(0, idx, s["k_new"].float(), "amin")
        hi = hi.scatter_reduce(0, idx, s["k_new"].float(), "amax")
        s["summary"].copy_(torch.stack([lo, hi], 2))
    return _store_out(s)


def _store_out(s):
    return {k: s[k] for k in ("k", "v", "summary")}


def _kept(lens, width, sink, recent):
    """Which of the positions 0 .. width - 1 each request's query sees."""
    j = torch.arange(width, device="cuda")[None]
    n = lens[:, None]
    keep = j < n
    if recent > 0:
        keep = keep & ((j < sink) | (j >= n - recent))
    return keep


def _decode_plain(s):
    c, lens, table = s["case"], s["seq_lens"].long(), s["block_table"].long()
    batch, h, d, dv = c["batch"], c["kv_heads"], c["dim"], s["dv"]
    group = c["q_heads"] // h
    width = table.shape[1] * PAGE
    keep = _kept(lens, width, c["sink"], c["recent"])
    k = s["k"][table].transpose(1, 2).reshape(batch, h, width, d).float()
    k.masked_fill_(~keep[:, None, :, None], 0.0)
    q = s["q"].float().reshape(batch, h, group, d)
    z = (q @ k.transpose(2, 3)) * s["sm_scale"]
    z.masked_fill_(~keep[:, None, None], -math.inf)
    if s["v"] is None:
        v = k[..., :dv]
    else:
        del k
        v = s["v"][table].transpose(1, 2).reshape(batch, h, width, dv).float()
        v.masked_fill_(~keep[:, None, :, None], 0.0)
    m = z.amax(3, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(3, keepdim=True)
    out = torch.where(l > 0, (p @ v) / l, torch.zeros((), device="cuda"))
    lse = torch.where(l > 0, m + torch.log(l), torch.full((), -math.inf, device="cuda"))
    s["out"].copy_(out.reshape(batch, h * group, dv))
    s["lse"].copy_(lse.reshape(batch, h * group))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import sparse_decode_attention_quest_gb300 as se
    op = s["case"]["op"]
    if op == "tables":
        se.se_block_tables_extend(s["free_pages"], s["pool_state"], s["block_table"], s["before"], s["new"],
                                  s["after"], s["token_start"], s["slot_map"], s["positions"])
        se.se_block_tables_release(s["free_pages"], s["pool_state"], s["block_table"], s["after"], s["before"])
        return _tables_out(s)
    if op == "store":
        se.se_paged_kv_store(s["kv"], s["k_new"], s["v_new"], s["slot_map"])
        return _store_out(s)
    se.se_paged_decode(s["kv"], s["q"], s["block_table"], s["seq_lens"], s["sm_scale"], s["out"], s["lse"],
                       s["workspace"], s["case"]["sink"], s["case"]["recent"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _tables_plain, "store": _store_plain, "decode": _decode_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def _mean_kept(lo, hi, sink, recent):
    """Tokens that a request's query sees, over lengths spread evenly between lo and hi."""
    n = [lo + (hi - lo) * i / 64 for i in range(65)]
    return sum(min(x, sink + recent) if recent > 0 else x for x in n) / len(n)


def work(case):
    batch = case["batch"]
    if case["op"] == "decode":
        h, hq, d = case["kv_heads"], case["q_heads"], case["dim"]
        dv = 512 if d == 576 else d
        kept = batch * _mean_kept(case["len_min"], case["len_max"], case["sink"], case["recent"])
        row = h * (d if d == 576 else d + dv) * 2
        return {"bytes": kept * (row + 4 / PAGE) + batch * (4 + hq * (2 * d + 2 * dv + 4)),
                "flops": 2.0 * kept * hq * (d + dv)}
    tokens = batch * (case["new_min"] + case["new_max"]) / 2
    opened = tokens / PAGE
    if case["op"] == "tables":
        # Lengths in and out, the slot and position arrays, every page from the stack to the
        # table and back.
        return {"bytes": 4 * (5 * batch + 2 * batch * case["new_max"] + 4 * opened), "flops": 4 * tokens}
    h, d = case["kv_heads"], case["dim"]
    rows = 2 * tokens * h * (1 if d == 576 else 2) * d * 2
    touched = max(opened, min(tokens, batch))
    return {"bytes": rows + 4 * tokens + (2 * touched * h * d * 2 if case["summary"] else 0),
            "flops": 2 * tokens * h * d if case["summary"] else 0}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run() returns, from the definitions: one request after another."""
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "store":
        slots = s["slot_map"].cpu()
        out = {"k": s["k"].double(), "v": None if s["v"] is None else s["v"].double(), "summary": None}
        at = slots.cuda().long()
        out["k"].transpose(1, 2)[at // PAGE, at % PAGE] = s["k_new"].double()
        if s["v"] is not None:
            out["v"].transpose(1, 2)[at // PAGE, at % PAGE] = s["v_new"].double()
        if s["summary"] is not None:
            # Over a page's slots: those written now, and the old bounds unless slot 0 is among them.
            written = torch.zeros(s["k"].shape[0] * PAGE, dtype=torch.bool)
            written[slots.long()] = True
            written = written.reshape(-1, 1, PAGE, 1).cuda()
            old = torch.where(written[:, :, :1], torch.tensor([math.inf, -math.inf]).cuda().double()[None, None, :, None],
                              s["summary"].double())
            lo = torch.where(written, out["k"], torch.full((), math.inf, dtype=torch.float64, device="cuda")).amin(2)
            hi = torch.where(written, out["k"], torch.full((), -math.inf, dtype=torch.float64, device="cuda")).amax(2)
            out["summary"] = torch.stack([torch.minimum(lo, old[:, :, 0]), torch.maximum(hi, old[:, :, 1])], 2)
        return out
    h, dv = case["kv_heads"], s["dv"]
    group = case["q_heads"] // h
    out = torch.zeros(case["batch"], case["q_heads"], dv, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        j = torch.arange(n, device="cuda")
        if case["recent"] > 0:
            j = torch.cat([j[:min(case["sink"], max(0, n - case["recent"]))], j[max(0, n - case["recent"]):]])
        if j.numel() == 0:
            continue
        page, slot = s["block_table"][b, j // PAGE].long(), j % PAGE
        keys = s["k"][page, :, slot].double()                      # [n][h][d]
        vals = keys[..., :dv] if s["v"] is None else s["v"][page, :, slot].double()
        q = s["q"][b].double().reshape(h, group, -1)
        z = s["sm_scale"] * torch.einsum("hgd,nhd->hgn", q, keys)
        lse[b] = torch.logsumexp(z, 2).reshape(-1)
        w = torch.exp(z - lse[b].reshape(h, group, 1))
        out[b] = torch.einsum("hgn,nhd->hgd", w, vals).reshape(-1, dv)
    return {"out": out, "lse": lse}
