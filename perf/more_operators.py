"""The 8-bit side of a paged KV cache, measured: rotary positions for the rows of new tokens, those rows
quantised into their pages, read back, and attended to.

Four operators, in the order a serving step uses them:

* ``rotary``  se_rotary: query and key rows turned by their tokens' positions (half and interleaved layouts,
  part of the head, frequencies scaled for long contexts, padded batches).
* ``store``   se_paged_kv8_store: the K and V rows of a ragged batch of new tokens into their slots as e4m3,
  with one scale for each page of 16 tokens and KV head.
* ``load``    se_paged_kv8_load: the rows of whole requests, or of a part of each, back as bf16.
* ``decode``  se_paged_kv8_decode: softmax(sm_scale q k) v of one query token per request over its cached
  tokens, all of them or the first ``sink`` and the last ``recent``.

``own`` chooses between the plain form (torch operations in fp32; angles in 64 bits) and the library's calls.
"""
import math

import torch

own = False

PAGE = 16
F8 = torch.float8_e4m3fn
LARGEST = 448.0          # of e4m3
LEAST_SCALE = 2.0 ** -100  # of a page of zeros


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The projections of one decode step: 32 requests at 64K-128K tokens.
        _rotary("rotary_decode_b32", batch=32, before=(65536, 131072), new=(1, 1), heads=(32, 4), dim=128, rot=128),
        # Four 32K prompts, read out of the fused QKV projection's output, with the smoothly scaled frequencies of a
        # context four times as long as the one trained for.
        _rotary("rotary_prefill_b4_32k", batch=4, before=(0, 0), new=(32768, 32768), heads=(32, 8), dim=128, rot=128,
                scaling="yarn", factor=4.0, original=32768),
        # Prompt chunks of odd lengths in a padded batch, for a latent cache: the last 64 of 576 dims, in place.
        _rotary("rotary_latent_b9", batch=9, before=(1, 200001), new=(1, 1501), heads=(64, 1), dim=576, rot=64,
                offset=512, interleaved=True, in_place=True, pad=237),
        # The rows of one decode step of 32 requests (4 KV heads).
        _store("store_decode_b32", batch=32, inside=True, new=(1, 1), heads=(32, 4), dim=128),
        # Four 32K prompts, 8 KV heads, read out of the fused projection's output.
        _store("store_prefill_b4_32k", batch=4, inside=False, new=(32768, 32768), heads=(32, 8), dim=128),
        # Prompt chunks of odd lengths that begin and end inside pages, heads of 256 dims.
        _store("store_chunks_b9", batch=9, inside=True, new=(1, 15001), heads=(16, 2), dim=256),
        # One request's history for the next chunk of its prompt.
        _load("load_b1_2k", batch=1, first=(0, 0), rows=(2049, 2049), kv_heads=4, dim=128),
        # Ragged spans of 13 requests (a prefix moved into a bf16 cache).
        _load("load_b13_32k", batch=13, first=(0, 3001), rows=(0, 32768), kv_heads=8, dim=128),
        # The smallest decode: one request, 4,096 tokens, one KV head.
        _decode("decode_b1_g4_4k", batch=1, lens=(4096, 4096), heads=(4, 1), dim=128),
        # Sink and recent windows over ragged histories, some requests still empty.
        _decode("decode_window_b48", batch=48, lens=(0, 33001), heads=(32, 4), dim=128, sink=64, recent=1000),
        # 32K contexts, 8 KV heads.
        _decode("decode_b8_32k", batch=8, lens=(32768, 32768), heads=(32, 8), dim=128),
        # Ragged 64K-128K contexts, 32 requests.
        _decode("decode_b32_128k", batch=32, lens=(65536, 131072), heads=(32, 4), dim=128),
    ]


def _rotary(name, batch, before, new, heads, dim, rot, offset=0, interleaved=False, scaling="none", factor=1.0,
            original=0, in_place=False, inverse=False, pad=0):
    """``heads``: query and key heads; ``pad``: rows behind the batch's last token."""
    return {"name": name, "op": "rotary", "batch": batch, "before_min": before[0], "before_max": before[1],
            "new_min": new[0], "new_max": new[1], "q_heads": heads[0], "kv_heads": heads[1], "dim": dim, "rot": rot,
            "offset": offset, "interleaved": interleaved, "scaling": scaling, "factor": factor, "original": original,
            "in_place": in_place, "inverse": inverse, "pad": pad}


def _store(name, batch, inside, new, heads, dim):
    """``inside``: requests already hold tokens, so that their first new one may land inside a page."""
    return {"name": name, "op": "store", "batch": batch, "inside": inside, "new_min": new[0], "new_max": new[1],
            "q_heads": heads[0], "kv_heads": heads[1], "dim": dim}


def _load(name, batch, first, rows, kv_heads, dim, pad=0):
    """``first``: the position that a request's rows begin at."""
    return {"name": name, "op": "load", "batch": batch, "first_min": first[0], "first_max": first[1],
            "rows_min": rows[0], "rows_max": rows[1], "kv_heads": kv_heads, "dim": dim, "pad": pad}


def _decode(name, batch, lens, heads, dim, sink=0, recent=0):
    return {"name": name, "op": "decode", "batch": batch, "len_min": lens[0], "len_max": lens[1], "q_heads": heads[0],
            "kv_heads": heads[1], "dim": dim, "sink": sink, "recent": recent}


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotary", "store", "load", "decode", "decode"])
    if op == "rotary":
        q, k, dim, rot, offset, interleaved = rng.choice([
            (32, 4, 128, 128, 0, False), (32, 8, 128, 64, 0, False), (28, 4, 128, 128, 0, True), (4, 1, 128, 96, 16, False),
            (12, 4, 64, 64, 0, False), (9, 3, 64, 32, 32, True), (16, 8, 256, 256, 0, False), (8, 1, 256, 64, 0, True),
            (10, 10, 128, 72, 0, False), (64, 1, 576, 64, 512, True), (16, 1, 576, 64, 512, False)])
        batch = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, min(32768, 1_300_000_000 // ((q + k) * dim * 2) // batch)))
        before = rng.choice([0, _log(rng, 1, 1_000_000)])
        scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 2.5), ("yarn", 32.0)])
        c = _rotary("", batch, (before // 2, before), (rng.choice([1, new]), new), (q, k), dim, rot, offset, interleaved,
                    scaling, factor, rng.choice([4096, 8192, 32768]), rng.random() < 0.5, rng.random() < 0.2,
                    rng.choice([0, 1, _log(rng, 1, 500)]))
    elif op in ("store", "load"):
        q, h, dim = rng.choice([(4, 1, 128), (12, 2, 128), (32, 4, 128), (32, 8, 128), (9, 3, 128), (0, 8, 64),
                                (5, 5, 64), (16, 4, 256), (8, 1, 256), (3, 3, 256)])
        batch = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, min(32768, (131072 * 1024 // (max(h, 4) * dim)) // batch)))
        if op == "store":
            c = _store("", batch, rng.random() < 0.7, (rng.choice([1, new]), new), (q, h), dim)
        else:
            c = _load("", batch, (0, rng.choice([0, _log(rng, 1, 8000)])), (rng.choice([0, 1, new]), new), h, dim,
                      rng.choice([0, 1, _log(rng, 1, 500)]))
    else:
        # Query and KV heads: groups of 1 to 64, KV head counts that are no power of two among them.
        q, h, dim = rng.choice([(4, 1, 128), (8, 8, 128), (16, 2, 128), (32, 8, 128), (32, 4, 128), (28, 4, 128),
                                (40, 8, 128), (10, 10, 128), (9, 3, 128), (32, 1, 128), (64, 1, 128), (64, 8, 64),
                                (12, 4, 64), (5, 5, 64), (16, 1, 64), (16, 8, 256), (8, 1, 256), (24, 2, 256)])
        longest = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(256, 3_200_000_000 // (2 * h * dim * longest))))
        sink, recent = (0, 0) if rng.random() < 0.6 else (rng.choice([0, 4, 64, _log(rng, 1, 500)]), _log(rng, 1, 4096))
        c = _decode("", batch, (rng.choice([0, 1, longest // 2, longest]), longest), (q, h), dim, sink, recent)
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


def _starts(n):
    return torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])


def _scale_of(amax):
    """The least power of two s with amax <= 448 s, and no less than LEAST_SCALE."""
    m, e = torch.frexp(amax)  # 448 is 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -100)).clamp_min(-100)
    return ((e + 127) << 23).view(torch.float32)


def _held(shape, g, channels=None):
    """Pages of normal values as a cache holds them: e4m3 and a scale for each page and head."""
    codes = torch.empty(shape, dtype=F8, device="cuda")
    scale = torch.empty(shape[:2], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        x = _normal((min(step, shape[0] - i),) + tuple(shape[1:]), g)
        if channels is not None:
            x.mul_(channels)
        s = _scale_of(x.abs().amax((2, 3)).float())
        scale[i:i + step] = s
        codes[i:i + step] = (x.float() / s[:, :, None, None]).to(F8)
    return codes, scale


def _loud_channels(h, d, g):
    """A few key channels per head are larger than the others, as in real caches."""
    scale = torch.ones(h, 1, d, dtype=torch.bfloat16)
    for i in range(h):
        scale[i, 0, torch.randperm(d, generator=g)[:4]] = 4.0
    return scale.cuda()


def _view(s):
    import sparse_decode_attention_quest_gb300 as se
    return se.paged_kv8(s["k"], s["v"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    dg = torch.Generator("cuda").manual_seed(seed)
    return {"rotary": _prepare_rotary, "store": _prepare_store, "load": _prepare_load,
            "decode": _prepare_decode}[case["op"]](case, g, dg)


def _prepare_rotary(case, g, dg):
    batch, hq, h, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    new = _lengths(case["new_min"], case["new_max"], batch, g)
    before = _lengths(case["before_min"], case["before_max"], batch, g)
    tokens = int(new.sum())
    r = torch.repeat_interleave(torch.arange(batch), new)
    rows = batch * case["new_max"] + case["pad"]  # what the program's buffers hold
    positions = torch.zeros(rows, dtype=torch.int32)
    positions[:tokens] = (before[r] + torch.arange(tokens) - (torch.cumsum(new, 0) - new)[r]).int()
    # Query and key rows: columns of the fused projection's output (the values behind them where there are any).
    fused = _normal((rows, hq + (1 if d == 576 else 2) * h, d), dg)
    s = {"case": case, "q": fused[:, :hq], "k": fused[:, hq:hq + h], "positions": positions.cuda(),
         "valid": torch.tensor([tokens], dtype=torch.int32, device="cuda")}
    s["q_out"] = s["q"] if case["in_place"] else torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = s["k"] if case["in_place"] else torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda")
    if own:  # the frequencies that a program keeps
        import sparse_decode_attention_quest_gb300 as se
        freqs, s["amplitude"] = se.se_rotary_frequencies(case["rot"], 10000.0, case["scaling"], case["factor"],
                                                         case["original"])
        s["freqs"] = freqs.cuda()
    else:
        inv, s["amplitude"] = _frequencies(case)
        s["inv_freq"] = inv.cuda()
    return s


def _frequencies(case):
    """Radians per position of each pair of dims, in 64 bits, and what cosines and sines are multiplied by."""
    rot, factor = case["rot"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = torch.tensor(10000.0, dtype=torch.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        inv = inv / factor
    if case["scaling"] != "yarn":
        return inv, 1.0
    # Pairs that turn more than 32 times over the original length stay, those under one turn are slowed by the factor.
    turns = case["original"] * inv / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return inv * keep + inv / factor * (1 - keep), 0.1 * math.log(factor) + 1


def _prepare_store(case, g, dg):
    batch, hq, h, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    new = _lengths(case["new_min"], case["new_max"], batch, g)
    # The pool holds the pages that take new tokens, in any order.
    inside = _lengths(0, PAGE - 1, batch, g) if case["inside"] else torch.zeros_like(new)
    tokens = int(new.sum())
    width = _pages((PAGE - 1 if case["inside"] else 0) + case["new_max"])
    pages = batch * width
    table = _paged(inside + new, torch.randperm(pages, generator=g), width)
    r = torch.repeat_interleave(torch.arange(batch), new)
    pos = inside[r] + torch.arange(tokens) - (torch.cumsum(new, 0) - new)[r]
    s = {"case": case, "slot_map": (table[r, pos // PAGE] * PAGE + (pos % PAGE).int()).int().cuda()}
    s["k"], s["k_scale"] = _held((pages, h, PAGE, d), dg)
    s["v"], s["v_scale"] = _held((pages, h, PAGE, d), dg)
    # Key and value rows: columns of the fused projection's output (the queries before them). Tokens differ in size, so
    # that some pages have to take a larger scale.
    fused = _normal((tokens, hq + 2 * h, d), dg)
    fused.mul_(torch.exp2(torch.randint(-2, 3, (tokens, 1, 1), generator=g).float()).bfloat16().cuda())
    s["k_new"], s["v_new"] = fused[:, hq:hq + h], fused[:, hq + h:]
    if own:
        s["kv"] = _view(s)
    return s


def _prepare_load(case, g, dg):
    batch, h, d = case["batch"], case["kv_heads"], case["dim"]
    rows = _lengths(case["rows_min"], case["rows_max"], batch, g)
    first = _lengths(case["first_min"], case["first_max"], batch, g)
    lens = first + rows
    total = max(1, int(_pages(lens).sum()))
    width = max(1, int(_pages(lens).max()))
    s = {"case": case, "block_table": _paged(lens, torch.randperm(total, generator=g), width).cuda(),
         "first": first.int().cuda() if case["first_max"] > 0 else None, "token_start": _starts(rows).int().cuda()}
    s["k"], s["k_scale"] = _held((total, h, PAGE, d), dg)
    s["v"], s["v_scale"] = _held((total, h, PAGE, d), dg)
    n = batch * case["rows_max"] + case["pad"]  # what the program's buffers hold
    s["k_out"] = torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda")
    s["v_out"] = torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda")
    if own:
        s["kv"] = _view(s)
    return s


def _prepare_decode(case, g, dg):
    batch, hq, h, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case["len_min"], case["len_max"], batch, g)
    total = max(1, int(_pages(lens).sum()))
    width = max(1, int(_pages(lens).max()))
    table = _paged(lens, torch.randperm(total, generator=g), width)
    s = {"case": case, "block_table": table.cuda(), "seq_lens": lens.int().cuda(), "sm_scale": 1.0 / math.sqrt(d)}
    s["k"], s["k_scale"] = _held((total, h, PAGE, d), dg, _loud_channels(h, d, g))
    s["v"], s["v_scale"] = _held((total, h, PAGE, d), dg)
    # What lies behind a request's last token in its last page is stale: NaN here.
    last = (lens - 1).clamp_min(0) // PAGE
    phys = table.long()[torch.arange(batch), last]
    slot = torch.arange(PAGE)
    stale = (slot[None] >= (lens - last * PAGE)[:, None]) & (lens > 0)[:, None]
    pi, si = (x.cuda() for x in (phys[:, None].expand(-1, PAGE)[stale], slot[None].expand(batch, -1)[stale]))
    for name in ("k", "v"):
        s[name].view(torch.uint8)[pi, :, si] = 0x7f
    s["q"] = _normal((batch, hq, d), dg)
    s["out"] = torch.empty(batch, hq, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(batch, hq, dtype=torch.float32, device="cuda")
    if own:  # the cache view and the workspace that a program keeps
        import sparse_decode_attention_quest_gb300 as se
        s["kv"] = _view(s)
        ws = se.se_paged_kv8_decode_workspace_size(batch, hq, h, d)
        s["workspace"] = torch.zeros(ws, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _rotary_plain(s):
    c = s["case"]
    rot, off = c["rot"], c["offset"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    if c["inverse"]:
        angle = -angle
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["amplitude"]).float()[:, None]
    live = (torch.arange(angle.shape[0], device="cuda") < s["valid"])[:, None, None]
    return {"q": _turned(s["q"], s["q_out"], cos, sin, live, rot, off, c["interleaved"]),
            "k": _turned(s["k"], s["k_out"], cos, sin, live, rot, off, c["interleaved"])}


def _turned(x, out, cos, sin, live, rot, off, interleaved):
    part = x[..., off:off + rot].float()
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y0, y1], 3).flatten(2) if interleaved else torch.cat([y0, y1], 2)
    whole = torch.cat([x[..., :off], y.bfloat16(), x[..., off + rot:]], 2)
    out.copy_(torch.where(live, whole, out))
    return out


def _store_plain(s):
    slot = s["slot_map"].long()
    page, off = slot // PAGE, slot % PAGE
    pages = s["k"].shape[0]
    fresh = torch.zeros(pages, dtype=torch.int32, device="cuda").scatter_reduce(0, page, (off == 0).int(), "amax") > 0
    _store_one(s["k"], s["k_scale"], s["k_new"], page, off, fresh)
    _store_one(s["v"], s["v_scale"], s["v_new"], page, off, fresh)
    return _store_out(s)


def _store_one(cache, scale, new, page, off, fresh):
    x = new.float()
    row = x.abs().amax(2)
    most = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(row), row, "amax")
    touched = torch.zeros_like(fresh).index_fill(0, page, True)
    old = torch.where(fresh[:, None], torch.zeros_like(scale), scale)
    grown = torch.where(touched[:, None], torch.maximum(old, _scale_of(most)), scale)
    # Rows of pages that take a larger scale are moved to it; rows of a page begun anew are whatever they were.
    ratio = torch.where((touched & ~fresh)[:, None], scale / grown, torch.ones_like(scale))
    cache.copy_((cache.float() * ratio[:, :, None, None]).to(F8))
    scale.copy_(grown)
    cache.view(torch.uint8)[page, :, off] = (x / grown[page][:, :, None]).to(F8).view(torch.uint8)


def _store_out(s):
    return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}


def _load_plain(s):
    start, table = s["token_start"].long(), s["block_table"].long()
    n = s["k_out"].shape[0]
    t = torch.arange(n, device="cuda")
    live = t < start[-1]
    r = torch.searchsorted(start[1:], t, right=True).clamp_max(table.shape[0] - 1)
    pos = t - start[r] + (0 if s["first"] is None else s["first"].long()[r])
    pos = torch.where(live, pos, torch.zeros_like(pos))
    page, off = table[r, pos // PAGE], pos % PAGE
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8)[page, :, off].view(F8).float()
        rows = codes * s[name + "_scale"][page][:, :, None]
        s[name + "_out"].copy_(torch.where(live[:, None, None], rows.bfloat16(), s[name + "_out"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _kept(lens, width, sink, recent):
    """Which of the positions 0 .. width - 1 each request's query sees."""
    j = torch.arange(width, device="cuda")[None]
    n = lens[:, None]
    keep = j < n
    if recent > 0:
        keep = keep & ((j < sink) | (j >= n - recent))
    return keep


def _rows_of(s, name, table, keep):
    """The rows of every request [batch][heads][width][dim] in fp32, 0 where they are not kept."""
    batch, width = keep.shape
    h, d = s[name].shape[1], s[name].shape[3]
    x = s[name].view(torch.uint8)[table].view(F8).float()
    x.mul_(s[name + "_scale"][table][..., None, None])
    x = x.transpose(1, 2).reshape(batch, h, width, d)
    return x.masked_fill_(~keep[:, None, :, None], 0.0)


def _decode_plain(s):
    c, lens, table = s["case"], s["seq_lens"].long(), s["block_table"].long()
    batch, hq, h, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    keep = _kept(lens, table.shape[1] * PAGE, c["sink"], c["recent"])
    q = s["q"].float().reshape(batch, h, hq // h, d)
    z = (q @ _rows_of(s, "k", table, keep).transpose(2, 3)) * s["sm_scale"]
    z.masked_fill_(~keep[:, None, None], -math.inf)
    m = z.amax(3, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(3, keepdim=True)
    out = torch.where(l > 0, (p @ _rows_of(s, "v", table, keep)) / l, torch.zeros((), device="cuda"))
    lse = torch.where(l > 0, m + torch.log(l), torch.full((), -math.inf, device="cuda"))
    s["out"].copy_(out.reshape(batch, hq, d))
    s["lse"].copy_(lse.reshape(batch, hq))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import sparse_decode_attention_quest_gb300 as se
    c = s["case"]
    if c["op"] == "rotary":
        q_out, k_out = (None, None) if c["in_place"] else (s["q_out"], s["k_out"])
        se.se_rotary(s["q"], s["k"], s["positions"], s["freqs"], q_out, k_out, rotary_offset=c["offset"],
                     interleaved=c["interleaved"], inverse=c["inverse"], amplitude=s["amplitude"],
                     num_valid=s["valid"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "store":
        se.se_paged_kv8_store(s["kv"], s["k_new"], s["v_new"], s["slot_map"])
        return _store_out(s)
    if c["op"] == "load":
        se.se_paged_kv8_load(s["kv"], s["block_table"], s["token_start"], s["k_out"], s["v_out"], s["first"])
        return {"k": s["k_out"], "v": s["v_out"]}
    se.se_paged_kv8_decode(s["kv"], s["q"], s["block_table"], s["seq_lens"], s["sm_scale"], s["out"], s["lse"],
                           s["workspace"], c["sink"], c["recent"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rotary": _rotary_plain, "store": _store_plain, "load": _load_plain,
            "decode": _decode_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def _mean_kept(lo, hi, sink, recent):
    """Tokens that a request's query sees, over lengths spread evenly between lo and hi."""
    n = [lo + (hi - lo) * i / 64 for i in range(65)]
    return sum(min(x, sink + recent) if recent > 0 else x for x in n) / len(n)


def work(case):
    batch, h, d = case["batch"], case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        tokens = batch * (case["new_min"] + case["new_max"]) / 2
        heads = case["q_heads"] + h
        width = case["rot"] if case["in_place"] else d
        return {"bytes": tokens * (heads * width * 4 + 4) + 8 * case["rot"] / 2, "flops": tokens * heads * case["rot"] * 3}
    if case["op"] == "store":
        tokens = batch * (case["new_min"] + case["new_max"]) / 2
        touched = max(tokens / PAGE, min(tokens, batch))
        return {"bytes": tokens * (2 * h * d * 3 + 4) + 2 * touched * h * 4, "flops": tokens * 2 * h * d * 2}
    if case["op"] == "load":
        rows = batch * (case["rows_min"] + case["rows_max"]) / 2
        return {"bytes": rows * (2 * h * (d * 3 + 4 / PAGE) + 4 / PAGE), "flops": rows * 2 * h * d}
    hq = case["q_heads"]
    kept = batch * _mean_kept(case["len_min"], case["len_max"], case["sink"], case["recent"])
    return {"bytes": kept * (2 * h * (d + 4 / PAGE) + 4 / PAGE) + batch * (4 + hq * (4 * d + 4)),
            "flops": 4.0 * kept * hq * d}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run() returns, from the definitions."""
    s = prepare(case, seed)
    return {"rotary": _rotary_exact, "store": _store_exact, "load": _load_exact, "decode": _decode_exact}[case["op"]](s)


def _rotary_exact(s):
    c = s["case"]
    rot, f = c["rot"], c["factor"]
    valid = int(s["valid"])
    pos = s["positions"][:valid].double()
    out = {"q": s["q_out"].double().clone(), "k": s["k_out"].double().clone()}
    for name in out:
        if not c["in_place"]:
            out[name][:valid] = s[name][:valid].double()
    for i in range(rot // 2):  # one pair of dims after another
        base = 10000.0 * f ** (rot / (rot - 2.0)) if c["scaling"] == "ntk" and rot > 2 else 10000.0
        w, size = math.exp(-2.0 * i / rot * math.log(base)), 1.0
        if c["scaling"] == "linear":
            w /= f
        if c["scaling"] == "yarn":
            keep = min(1.0, max(0.0, (c["original"] * w / (2 * math.pi) - 1.0) / 31.0))
            w, size = (1 - keep) * w / f + keep * w, 1.0 + 0.1 * math.log(f)
        turn = torch.polar(torch.full_like(pos, size), pos * (-w if c["inverse"] else w))[:, None]
        i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
        for name in out:
            x = s[name][:valid].double()
            y = torch.complex(x[..., c["offset"] + i0], x[..., c["offset"] + i1]) * turn
            out[name][:valid, :, c["offset"] + i0] = y.real
            out[name][:valid, :, c["offset"] + i1] = y.imag
    return out


def _to_e4m3(y):
    """The nearest value of e4m3 (ties to even), for |y| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _store_exact(s):
    if s["slot_map"].numel() * s["case"]["kv_heads"] * s["case"]["dim"] > 1 << 28:
        return None
    slots = s["slot_map"].long()
    pages = s["k"].shape[0]
    written = torch.zeros(pages * PAGE, dtype=torch.bool, device="cuda")
    written[slots] = True
    written = written.reshape(pages, 1, PAGE, 1)
    any_new, opened = written.any(2)[..., 0], written[:, :, 0, 0]
    out = {}
    for name in ("k", "v"):
        x = torch.zeros(pages, PAGE, *s[name + "_new"].shape[1:], dtype=torch.float64, device="cuda")
        x.view(-1, *x.shape[2:])[slots] = s[name + "_new"].double()
        x = x.transpose(1, 2)
        amax = (x * written).abs().amax((2, 3))
        need = torch.full_like(amax, LEAST_SCALE)
        for _ in range(240):
            need = torch.where(amax > LARGEST * need, 2 * need, need)
        old = s[name + "_scale"].double()
        scale = torch.where(any_new, torch.where(opened, need, torch.maximum(old, need)), old)
        codes = s[name].double()
        moved = torch.where(opened[..., None, None], codes, _to_e4m3(codes * (old / scale)[..., None, None]))
        out[name] = torch.where(written, _to_e4m3(x / scale[..., None, None]), moved)
        out[name + "_scale"] = scale
    return out


def _load_exact(s):
    out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
    start = s["token_start"].tolist()
    for b in range(s["case"]["batch"]):
        j = torch.arange(start[b + 1] - start[b], device="cuda")
        if s["first"] is not None:
            j = j + int(s["first"][b])
        page, slot = s["block_table"][b, j // PAGE].long(), j % PAGE
        for name in ("k", "v"):
            codes = s[name].view(torch.uint8)[page, :, slot].view(F8).double()
            out[name][start[b]:start[b + 1]] = codes * s[name + "_scale"][page].double()[..., None]
    return out


def _decode_exact(s):
    case = s["case"]
    h, d = case["kv_heads"], case["dim"]
    group = case["q_heads"] // h
    out = torch.zeros(case["batch"], case["q_heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        j = torch.arange(n, device="cuda")
        if case["recent"] > 0:
            j = torch.cat([j[:min(case["sink"], max(0, n - case["recent"]))], j[max(0, n - case["recent"]):]])
        if j.numel() == 0:
            continue
        page, slot = s["block_table"][b, j // PAGE].long(), j % PAGE
        held = [s[x].view(torch.uint8)[page, :, slot].view(F8).double() * s[x + "_scale"][page].double()[..., None]
                for x in ("k", "v")]                                     # [n][h][d]
        q = s["q"][b].double().reshape(h, group, d)
        z = s["sm_scale"] * torch.einsum("hgd,nhd->hgn", q, held[0])
        lse[b] = torch.logsumexp(z, 2).reshape(-1)
        w = torch.exp(z - lse[b].reshape(h, group, 1))
        out[b] = torch.einsum("hgn,nhd->hgd", w, held[1]).reshape(-1, d)
    return {"out": out, "lse": lse}
