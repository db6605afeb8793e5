"""The operators around a key/value cache held in 4 bits, as they are measured: cases, inputs,
plain forms in elementary torch operations, and the calls of the package's own kernels.

  plan       page tables, slots and positions of a serving step from the requests' lengths
  append     rotary positions on q and k, and k and v rounded to 4 bits into their slots; the
             rows are read back as the values they stand for
  read       rows of the cache as the values they stand for
  attention  softmax attention of new tokens over the paged cache

A cache page holds, for each of the kv heads, page_tokens / 16 tiles of 16 tokens. A tile is the
keys' quants, the keys' scales, the values' quants and the values' scales. A row of head_dim
values is head_dim / 32 blocks; block b stands for d * (n - 8), d in fp16, n in 0..15. A byte of
quants holds the block's values i (low half) and i + 16 (high half), i < 16.
  keys    [chunk][i / 4][token][word][byte]      block = chunk * words + word, byte P[i % 4]
  values  [chunk][token / 4][i][word][byte]      byte P[token % 4]
  scales  [token / 4][block][token % 4]          fp16
with P = (0, 2, 1, 3), and `words` the blocks of a chunk: all of them up to 4, else 4.
"""
import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # a few requests, each one token further: the start of every decode step
        {"name": "plan decode 8", "op": "plan", "requests": 8, "rows": 8, "max_len": 4096,
         "prompt": 1, "page_tokens": 64},
        # a full server: ended requests give their pages back, new prompts come in beside decodes
        {"name": "plan mixed 512", "op": "plan", "requests": 512, "rows": 16384, "max_len": 8192,
         "prompt": 240, "page_tokens": 16},
        # one token of one sequence (the 8B-shaped decode step's q, k and v rows)
        {"name": "append 1 f32", "op": "append", "rows": 1, "pad": 0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "page_tokens": 64, "max_pos": 4096, "axes": 1,
         "rot": 128, "interleaved": False, "dtype": "f32"},
        # images and text in one batch: three position axes, an odd count, rows of padding
        {"name": "append 1501 f16 axes", "op": "append", "rows": 1501, "pad": 35, "q_heads": 16,
         "kv_heads": 16, "head_dim": 64, "page_tokens": 16, "max_pos": 100000, "axes": 3,
         "rot": 64, "interleaved": True, "dtype": "f16"},
        # a prompt of the 70B-shaped layer
        {"name": "append 8192 bf16", "op": "append", "rows": 8192, "pad": 0, "q_heads": 64,
         "kv_heads": 8, "head_dim": 128, "page_tokens": 64, "max_pos": 32768, "axes": 1,
         "rot": 128, "interleaved": False, "dtype": "bf16"},
        # a short prefix taken out of the cache at full precision
        {"name": "read 777 f32", "op": "read", "rows": 777, "kv_heads": 8, "head_dim": 128,
         "page_tokens": 16, "dtype": "f32"},
        # a long shared prefix, moved to another cache or another kernel
        {"name": "read 65536 bf16", "op": "read", "rows": 65536, "kv_heads": 8, "head_dim": 128,
         "page_tokens": 64, "dtype": "bf16"},
        # one sequence, one token, the framework's own activation type
        {"name": "attention 1x4096 f32", "op": "attention", "requests": 1, "new": 1, "min_len": 4096,
         "max_len": 4096, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page_tokens": 64,
         "window": 0, "dtype": "f32"},
        # a decode batch of very different lengths
        {"name": "attention 64x8192 bf16", "op": "attention", "requests": 64, "new": 1,
         "min_len": 1, "max_len": 8192, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "page_tokens": 64, "window": 0, "dtype": "bf16"},
        # one very long context
        {"name": "attention 1x131072 f16", "op": "attention", "requests": 1, "new": 1,
         "min_len": 131072, "max_len": 131072, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page_tokens": 16, "window": 0, "dtype": "f16"},
        # drafted tokens checked in one pass, a sliding window, odd lengths
        {"name": "attention 24x5 window f16", "op": "attention", "requests": 24, "new": 5,
         "min_len": 5, "max_len": 5000, "q_heads": 16, "kv_heads": 4, "head_dim": 256,
         "page_tokens": 32, "window": 1111, "dtype": "f16"},
        # pieces of prompts over what is cached already
        {"name": "attention 4x1024 bf16", "op": "attention", "requests": 4, "new": 1024,
         "min_len": 1024, "max_len": 8192, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page_tokens": 64, "window": 0, "dtype": "bf16"},
    ]


def _between(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "read", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f32", "bf16", "f16"])
    dim = rng.choice([64, 96, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    if op == "plan":
        n = _between(rng, 1, 512)
        prompt = rng.choice([1, 1, _between(rng, 2, 240)])
        return {"op": op, "requests": n, "rows": n * prompt + rng.randrange(9),
                "max_len": _between(rng, 1, 8192), "prompt": prompt, "page_tokens": page}
    if op == "append":
        axes = rng.choice([1, 1, 2, 3])
        most = max(1, 8192 * 80 * 128 // (kv * (group + 2) * dim * 2))
        rot = rng.choice([dim, dim, dim // 2])
        return {"op": op, "rows": _between(rng, 1, min(8192, most)), "pad": rng.choice([0, 0, 7]),
                "q_heads": kv * group, "kv_heads": kv, "head_dim": dim, "page_tokens": page,
                "max_pos": _between(rng, 64, 1000000), "axes": axes, "rot": rot,
                "interleaved": rng.random() < 0.4, "dtype": dtype}
    if op == "read":
        most = max(1, 65536 * 8 * 128 // (kv * dim * 2))
        return {"op": op, "rows": _between(rng, 1, min(65536, most)), "kv_heads": kv,
                "head_dim": dim, "page_tokens": page, "dtype": dtype}
    kind = rng.choice(["decode", "decode", "draft", "prompt"])
    n = {"decode": _between(rng, 1, 64), "draft": _between(rng, 1, 24), "prompt": rng.randint(1, 3)}[kind]
    new = {"decode": 1, "draft": rng.randint(2, 8), "prompt": _between(rng, 16, 512)}[kind]
    if kind == "prompt":
        kv, group = min(kv, 8), min(group, 4)
    room = 64 * 8192 * 8 * 128 // (n * kv * dim * (2 if dtype == "f32" else 1))
    longest = max(new, min(8192 if n > 4 or kind == "prompt" else 100000, room))
    return {"op": op, "requests": n, "new": new, "min_len": rng.choice([new, longest]) if kind == "decode" else new,
            "max_len": max(new, _between(rng, max(1, longest // 64), longest)) if kind != "decode" else longest,
            "q_heads": kv * group, "kv_heads": kv, "head_dim": dim, "page_tokens": page,
            "window": rng.choice([0, 0, 0, _between(rng, 1, 4096)]), "dtype": dtype}


def _lengths(c):
    """The requests' lengths after the step and their new tokens, longest first: even steps from
    max_len down to min_len; the new tokens of a request are `new`, or fewer where new > 8 (pieces
    of prompts end anywhere)."""
    n, lo, hi, new = c["requests"], c["min_len"], c["max_len"], c["new"]
    lens = [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]
    news = [min(new if new <= 8 else max(1, new - i * new // (4 * n)), ln) for i, ln in enumerate(lens)]
    return lens, news


def _plan_lengths(c):
    """(tokens in the cache, new tokens) of each request of a plan case; new -1: it has ended."""
    n, hi, prompt = c["requests"], c["max_len"], c["prompt"]
    pairs, room = [], c["rows"]
    for i in range(n):
        ln = 1 + (hi - 1) * ((i * 37 + 11) % n) // max(1, n - 1) if n > 1 else hi
        if i % 16 == 15:
            pairs.append((ln, -1))
            continue
        new = 0 if i % 16 == 9 else 1
        if prompt > 1 and i % 4 == 2:  # a prompt, or a piece of one
            new = 1 + (prompt - 1) * (i % 13) // 12
            ln = 0 if i % 8 == 2 else ln
        new = min(new, room)
        room -= new
        pairs.append((ln, new))
    return pairs


# ---- what a program has in hand ----------------------------------------------------------------

def _words(dim):
    return min(dim // 32, 4)


def _tile_parts(dim):
    """Bytes of a tile's quants and scales, of the keys or of the values."""
    return 8 * dim, dim // 32 * 32


def _cache(c, pages, gen):
    """Pages with random quants and scales (values of unit size) on the GPU."""
    dim, kv = c["head_dim"], c["kv_heads"]
    quants, scales = _tile_parts(dim)
    tiles = (pages, kv, c["page_tokens"] // 16)
    data = torch.randint(0, 256, tiles + (2, quants + scales), dtype=torch.uint8, device="cuda", generator=gen)
    d = torch.rand(tiles + (2, scales // 2), device="cuda", generator=gen)
    d = (0.1 + 0.25 * d) * (1 - 2 * (d > 0.5))  # GGUF scales have either sign
    data[..., quants:] = d.half().view(torch.uint8)
    return data.view(pages, -1)


def _normal(shape, dtype, gen):
    return torch.randn(shape, device="cuda", generator=gen).to(_DTYPES[dtype])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c}
    P = c["page_tokens"]
    if c["op"] == "plan":
        pairs = _plan_lengths(c)
        rng.shuffle(pairs)
        R, mb = len(pairs), -(-(c["max_len"] + c["prompt"]) // P)
        have = [-(-ln // P) for ln, _ in pairs]
        pages = sum(have) + R * (1 + -(-c["prompt"] // P)) + 5
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((R, mb), -1, dtype=torch.int32, device="cuda")
        taken = torch.arange(mb, device="cuda")[None] < i32(have)[:, None]
        table[taken] = order[:sum(have)]
        free = torch.zeros(pages, dtype=torch.int32, device="cuda")
        free[:pages - sum(have)] = order[sum(have):]
        s.update(kv_len=i32([a for a, _ in pairs]), new_len=i32([b for _, b in pairs]), table=table,
                 free=free, free_count=i32([pages - sum(have)]), pages=pages,
                 # the plan takes no keys or values: the smallest cache of this page count
                 data=torch.empty((pages, 2 * (P // 16) * sum(_tile_parts(64))), dtype=torch.uint8, device="cuda"))
        return s
    if c["op"] == "attention":
        lens, news = _lengths(c)
        both = list(zip(lens, news))
        rng.shuffle(both)
        lens, news = [a for a, _ in both], [b for _, b in both]
        R, mb = len(lens), -(-max(lens) // P)
        have = [-(-ln // P) for ln in lens]
        pages = sum(have) + 3
        s["data"] = _cache(c, pages, gen)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.full((R, mb), -1, dtype=torch.int32, device="cuda")
        s["table"][torch.arange(mb, device="cuda")[None] < i32(have)[:, None]] = order[:sum(have)]
        s["seq_len"] = i32(lens)
        s["cu_new"] = i32([sum(news[:i]) for i in range(R + 1)])
        s["most_new"], s["most_len"] = max(news), max(lens)
        # queries with some reach: logits of about two
        q = 2.0 * torch.randn((sum(news), c["q_heads"], c["head_dim"]), device="cuda", generator=gen)
        s["q"] = q.to(_DTYPES[c["dtype"]])
        return s
    rows = c["rows"] + c.get("pad", 0)
    pages = -(-c["rows"] // P) + 3
    where = torch.randperm(pages, generator=gen, device="cuda")
    at = torch.arange(c["rows"], device="cuda") + rng.randrange(P)  # a request's rows start inside a page
    s["slots"] = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    s["slots"][:c["rows"]] = (where[at // P] * P + at % P).to(torch.int32)
    s["data"] = _cache(c, pages, gen)
    if c["op"] == "read":
        return s
    kv, dim = c["kv_heads"], c["head_dim"]
    # q, k and v as one projection's output: rows of one buffer
    qkv = _normal((rows, c["q_heads"] + 2 * kv, dim), c["dtype"], gen)
    s["q"], s["k"], s["v"] = qkv.split([c["q_heads"], kv, kv], dim=1)
    start = rng.randrange(c["max_pos"])
    pos = torch.randint(0, c["max_pos"], (c["axes"], rows), dtype=torch.int32, device="cuda", generator=gen)
    pos[0] = (start + torch.arange(rows, device="cuda")).remainder(c["max_pos"]).to(torch.int32)
    s["positions"] = pos
    pairs = c["rot"] // 2
    s["inv_freq"] = (500000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float()
    s["sections"] = [pairs // c["axes"] + (i < pairs % c["axes"]) for i in range(c["axes"])]
    s["q_out"] = torch.zeros((rows, c["q_heads"], dim), dtype=_DTYPES[c["dtype"]], device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"plan": _plan, "append": _append, "read": _read, "attention": _attention}[op](state)


def _own(s, op):
    import moe_expert_ffn_q4_amd as tq

    c = s["case"]
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside the cache's memory
        cache = s["cache"] = tq.KvCache(c.get("kv_heads", 1), c.get("head_dim", 64), c["page_tokens"], data=s["data"])
    if op == "plan":
        return tq.kv_plan(cache, s["kv_len"], s["new_len"], s["table"], c["rows"], s["free"], s["free_count"])
    if op == "read":
        return tq.kv_read(cache, s["slots"], _DTYPES[c["dtype"]])
    if op == "append":
        if "rope" not in s:
            s["rope"] = tq.Rope(s["inv_freq"], s["sections"], interleaved=c["interleaved"])
        q = tq.kv_append(cache, s["k"], s["v"], s["slots"], q=s["q"], rope=s["rope"], positions=s["positions"], q_out=s["q_out"])
        return (q,) + tuple(tq.kv_read(cache, s["slots"][:c["rows"]], _DTYPES[c["dtype"]]))
    return tq.kv_attention(cache, s["q"], s["table"], s["seq_len"], s["cu_new"], window=c["window"], return_lse=True)


def _plan(s):
    c, P = s["case"], s["case"]["page_tokens"]
    kv, new, table, free = s["kv_len"].long(), s["new_len"].long(), s["table"].long(), s["free"].long()
    R, mb = table.shape
    ended, n = new < 0, new.clamp(min=0)
    after = torch.where(ended, 0, kv + n)
    have = (kv + P - 1) // P
    need = torch.where(ended, 0, (after + P - 1) // P - have)
    back = torch.where(ended, have, 0)
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    col = torch.arange(mb, device=kv.device)[None]
    # the pages of ended requests go on top of the free list, in order
    count = s["free_count"].long()
    goes = ended[:, None] & (col < have[:, None])
    to = torch.where(goes, count + (back.cumsum(0) - back)[:, None] + col, free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, to.view(-1), table.view(-1))[:-1]
    top = count + back.sum()
    # needed pages come off the top, in order
    comes = (col >= have[:, None]) & (col < (have + need)[:, None])
    frm = top - 1 - ((need.cumsum(0) - need)[:, None] + col - have[:, None])
    table = torch.where(comes, stack[frm.clamp(0, free.numel() - 1)], table)
    t = torch.arange(c["rows"], device=kv.device)
    live = t < cu[-1]
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    pos = kv[r] + t - cu[r]
    slot = table[r, (pos // P).clamp(0, mb - 1)] * P + pos % P
    out = {"block_table": table, "cu_new": cu, "seq_len": after, "slots": torch.where(live, slot, -1),
           "positions": torch.where(live, pos, -1), "requests": torch.where(live, r, -1), "free_pages": stack,
           "free_count": top - need.sum(), "status": torch.zeros(1, device=kv.device)}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _unpack(tiles, dim):
    """Keys and values [..., 16, dim] in fp32 of tiles [..., 2, bytes]."""
    lead, nb, w = tiles.shape[:-2], dim // 32, _words(dim)
    quants, _ = _tile_parts(dim)
    byte = tiles[..., :quants].reshape(lead + (2, nb // w, 4, 16, w, 4))[..., [0, 2, 1, 3]]
    n = torch.stack([byte & 15, byte >> 4], -1)  # [kv, chunk, 4, 16, word, byte, half]
    d = tiles[..., quants:].contiguous().view(torch.float16).view(lead + (2, 4, nb, 4)).float()
    d = d.transpose(-1, -2).reshape(lead + (2, 16, nb, 1))
    a = len(lead)
    ax = list(range(a))
    k = n.select(a, 0).permute(ax + [a + 2, a, a + 3, a + 5, a + 1, a + 4]).reshape(lead + (16, nb, 32))
    v = n.select(a, 1).permute(ax + [a + 1, a + 4, a, a + 3, a + 5, a + 2]).reshape(lead + (16, nb, 32))
    k = (k.float() - 8) * d.select(a, 0)
    v = (v.float() - 8) * d.select(a, 1)
    return k.reshape(lead + (16, dim)), v.reshape(lead + (16, dim))


def _tiles(s):
    """The cache as [pages, kv heads, tiles, 2, bytes]."""
    c = s["case"]
    return s["data"].view(s["data"].shape[0], c["kv_heads"], c["page_tokens"] // 16, 2, sum(_tile_parts(c["head_dim"])))


def _read(s):
    c, P, slots = s["case"], s["case"]["page_tokens"], s["slots"].long()
    picked = _tiles(s)[slots // P, :, slots % P // 16]  # [rows, heads, 2, bytes]
    token = (slots % 16).view(-1, 1, 1, 1).expand(-1, c["kv_heads"], 1, c["head_dim"])
    k, v = _unpack(picked, c["head_dim"])
    return tuple(x.gather(2, token)[:, :, 0].to(_DTYPES[c["dtype"]]) for x in (k, v))


def _turn(x, s):
    """Rows x [rows, heads, dim] turned by their positions, in 64 bits."""
    c = s["case"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=x.device), torch.tensor(s["sections"], device=x.device), output_size=c["rot"] // 2)
    angle = (s["positions"].double()[axis] * s["inv_freq"].double()[:, None]).t()[:, None]
    co, si = angle.cos(), angle.sin()
    x = x.double()
    t = x[..., :c["rot"]]
    if c["interleaved"]:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
    else:
        a, b = t.chunk(2, -1)
        t = torch.cat([a * co - b * si, a * si + b * co], -1)
    return torch.cat([t, x[..., c["rot"]:]], -1)


def _round4(x):
    """Rows of fp32 as the values that their 4-bit blocks stand for."""
    x = x.unflatten(-1, (-1, 32))
    a = x.abs()
    most = a.amax(-1, keepdim=True)
    first = torch.where(a == most, torch.arange(32, device=x.device), 32).amin(-1, keepdim=True)
    d = (x.gather(-1, first) / -8).clamp(-65504, 65504).half().double()
    n = torch.where(d == 0, 0.0, torch.round(x.double() / torch.where(d == 0, 1.0, d))).clamp(-8, 7)
    return (n * d).float().flatten(-2)


def _append(s):
    c, n = s["case"], s["case"]["rows"]
    dt = _DTYPES[c["dtype"]]
    q = torch.zeros_like(s["q_out"])
    q[:n] = _turn(s["q"], s)[:n].to(dt)
    return q, _round4(_turn(s["k"], s)[:n].float()).to(dt), _round4(s["v"][:n].float()).to(dt)


def _attention(s):
    c, dim, P = s["case"], s["case"]["head_dim"], s["case"]["page_tokens"]
    kv, G, most = c["kv_heads"], c["q_heads"] // c["kv_heads"], s["most_new"]
    table, lens, cu = s["table"].long(), s["seq_len"].long(), s["cu_new"].long()
    R, mb = table.shape
    # every request's pages as rows of keys and values, padded to the longest
    k, v = _unpack(_tiles(s)[table.clamp(min=0)], dim)  # [R, mb, kv, tiles, 16, dim]
    k, v = (x.transpose(1, 2).reshape(R, kv, mb * P, dim) for x in (k, v))
    # the new tokens of every request, padded to the most
    i = torch.arange(most, device=k.device)
    news = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(R, most, kv, G, dim).permute(0, 2, 3, 1, 4).reshape(R, kv, G * most, dim)
    logits = torch.matmul(q * dim ** -0.5, k.transpose(-1, -2).contiguous()).view(R, kv, G, most, mb * P)
    pos = (lens - news)[:, None] + i
    t = torch.arange(mb * P, device=k.device)
    seen = t <= pos[..., None]
    if c["window"]:
        seen &= t > pos[..., None] - c["window"]
    logits = torch.where(seen[:, None, None], logits, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (logits - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(R, kv, G * most, -1), v).view(R, kv, G, most, dim) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    rows = torch.searchsorted(cu[1:], torch.arange(s["q"].shape[0], device=k.device), right=True)
    own_i = torch.arange(s["q"].shape[0], device=k.device) - cu[rows]
    out = out.permute(0, 3, 1, 2, 4).reshape(R, most, kv * G, dim)[rows, own_i]
    lse = lse.permute(0, 3, 1, 2).reshape(R, most, kv * G)[rows, own_i]
    return out.to(s["q"].dtype), lse


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _rows64(s, slots, which):
    """Rows of the cache in 64 bits, element by element from the layout's offsets."""
    c, dim = s["case"], s["case"]["head_dim"]
    P, kv, nb, w = c["page_tokens"], c["kv_heads"], dim // 32, _words(dim)
    quants, scales = _tile_parts(dim)
    flat, dev = s["data"].view(-1), s["data"].device
    slots = slots.long()[:, None, None]
    head = torch.arange(kv, device=dev)[None, :, None]
    e = torch.arange(dim, device=dev)[None, None]
    b, half, i = e // 32, e % 32 // 16, e % 16
    tok = slots % 16
    order = torch.tensor([0, 2, 1, 3], device=dev)
    base = ((slots // P * kv + head) * (P // 16) + slots % P // 16) * 2 * (quants + scales) + which * (quants + scales)
    word = lambda four, sixteen: (((b // w * 4 + four) * 16 + sixteen) * w + b % w) * 4  # noqa: E731
    at = word(i // 4, tok) + order[i % 4] if which == 0 else word(tok // 4, i) + order[tok % 4]
    n = (flat[base + at].long() >> (4 * half)) & 15
    d_at = base + quants + ((tok // 4 * nb + b) * 4 + tok % 4) * 2
    bits = flat[d_at].int() | flat[d_at + 1].int() << 8
    return (n - 8).double() * bits.to(torch.int16).view(torch.float16).double()


def _quantized64(x):
    """x [..., 32] fp32 rounded to a block: the largest magnitude (the first one) stands at -8."""
    at = (x.abs() == x.abs().max(-1, keepdim=True).values).int().cummax(-1).values.sum(-1, keepdim=True)
    d = torch.take_along_dim(x, 32 - at, -1).double().div(-8).clamp(-65504, 65504).to(torch.float16).double()
    ratio = torch.nan_to_num(x.double() / d, nan=0.0, posinf=0.0, neginf=0.0)
    return d * ratio.round().clamp(-8, 7)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "plan":
        return None
    if c["op"] == "read":
        return tuple(_rows64(s, s["slots"], w) for w in (0, 1))
    if c["op"] == "append":
        n, rot = c["rows"], c["rot"]
        axis = [a for a, m in enumerate(s["sections"]) for _ in range(m)]
        turned = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for p in range(rot // 2):
                th = s["positions"][axis[p]].double() * float(s["inv_freq"][p])
                i, j = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + rot // 2)
                z = torch.complex(x[..., i].double(), x[..., j].double()) * torch.polar(torch.ones_like(th), th)[:, None]
                y[..., i], y[..., j] = z.real, z.imag
            turned.append(y)
        q = torch.zeros_like(turned[0])
        q[:n] = turned[0][:n]
        k, v = turned[1][:n].float(), s["v"][:n].float()
        return (q,) + tuple(_quantized64(x.unflatten(-1, (-1, 32))).flatten(-2) for x in (k, v))
    P, dim, G = c["page_tokens"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    cu, lens = s["cu_new"].tolist(), s["seq_len"].tolist()
    for r, ln in enumerate(lens):
        t = torch.arange(ln, device="cuda")
        slots = s["table"][r].long()[t // P] * P + t % P
        k, v = (_rows64(s, slots, w) for w in (0, 1))
        new = cu[r + 1] - cu[r]
        pos = ln - new + torch.arange(new, device="cuda")
        hidden = t[None] > pos[:, None]
        if c["window"]:
            hidden |= t[None] <= pos[:, None] - c["window"]
        for h in range(c["q_heads"]):
            x = s["q"][cu[r]:cu[r + 1], h].double() @ k[:, h // G].t() / math.sqrt(dim)
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[cu[r]:cu[r + 1], h] = z
            out[cu[r]:cu[r + 1], h] = (x - z[:, None]).exp() @ v[:, h // G]
    return out, lse


# ---- what a pass cannot do without ------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "plan":
        pairs, P = _plan_lengths(c), c["page_tokens"]
        moved = sum(-(-a // P) if b < 0 else -(-(a + b) // P) - -(-a // P) for a, b in pairs)
        # lengths in, tables of the pages that move, the rows' slots, positions and requests out
        return {"bytes": 4 * (4 * len(pairs) + 2 * moved + 3 * c["rows"] + 4), "flops": 0}
    kv, dim, b = c["kv_heads"], c["head_dim"], _SIZE[c["dtype"]]
    row = 2 * kv * (dim // 2 + dim // 32 * 2)  # a token's keys and values in the cache
    if c["op"] == "read":
        return {"bytes": c["rows"] * (row + 4 + 2 * kv * dim * b), "flops": c["rows"] * 2 * kv * dim}
    if c["op"] == "append":
        n = c["rows"]
        acts = n * dim * b * (2 * c["q_heads"] + 2 * kv)  # q in and out, k and v in
        back = n * (row + 2 * kv * dim * b)  # the rows read back
        return {"bytes": acts + n * (row + 4 + 4 * c["axes"]) + back,
                "flops": n * dim * (3 * c["q_heads"] + 9 * kv)}
    lens, news = _lengths(c)
    read = seen = 0
    for ln, new in zip(lens, news):
        w = c["window"] or ln
        read += ln - max(0, ln - new - w + 1)
        first, last = ln - new + 1, ln  # keys that the first and the last new token see
        below = max(0, min(last, w) - first + 1)  # tokens that the window does not cut
        seen += below * (2 * first + below - 1) // 2 + (new - below) * w
    rows = sum(news)
    return {"bytes": read * row + rows * c["q_heads"] * (2 * dim * b + 4) + 4 * (2 * len(lens) + sum(-(-ln // c["page_tokens"]) for ln in lens)),
            "flops": 4 * dim * c["q_heads"] * seen}
