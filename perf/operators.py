"""The paged-cache operators: their plain forms, the library's calls, and the
cases both are measured on.

Four operators of a serving step over a K/V cache kept in pages:

  plan     block tables, slot map and positions of a step, from the requests'
           lengths (``Block.page_plan``)
  append   K/V rows into their pages by slot map (``Block.page_append``)
  attend   attention of a ragged batch over paged caches: one new token per
           sequence (decode), a few (drafts to verify) or many (prompt chunks)
           (``Block.attn_paged``)
  prefix   the same for a batch whose sequences share their first slots, the
           shared part computed once for all rows

With ``own`` false ``run`` is the plain form in elementary torch operations
(fp32, rounded once at the end); with ``own`` true it makes the library's calls.

Pools are [n_pages, kv_heads, page, dim] fp16.  Row t of sequence b sits in
slot cache_lens[b] + t and sees slots [0, cache_lens[b] + t].
"""
import math
import random

import torch

own = False

_DEV = "cuda"
_blocks = {}


# ---------------------------------------------------------------- cases
def _plan(name, B, lo, hi, new_lo, new_hi, page, mix):
    return {"name": name, "op": "plan", "B": B, "lo": lo, "hi": hi, "new_lo": new_lo,
            "new_hi": new_hi, "page": page, "mix": mix}


def _append(name, rows, kv_heads, dim, page, head_major):
    return {"name": name, "op": "append", "rows": rows, "kv_heads": kv_heads, "dim": dim,
            "page": page, "head_major": head_major}


def _attend(name, B, lo, hi, new_lo, new_hi, heads, kv_heads, dim, page, mix, prefix=0,
            packed=False):
    return {"name": name, "op": "prefix" if prefix else "attend", "B": B, "lo": lo, "hi": hi,
            "new_lo": new_lo, "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "mix": mix, "prefix": prefix, "packed": packed}


def listed():
    return [
        # one decode step of 64 requests near 1024 tokens: the batched decode's usual batch
        _plan("plan_decode_64", 64, 1000, 1030, 1, 1, 64, 1),
        # admission of 200 prompts of odd lengths at once, small pages
        _plan("plan_prompts_200", 200, 0, 40, 1, 999, 16, 2),
        # the K/V rows of one decode step of 64 requests
        _append("append_step_64", 64, 2, 128, 64, False),
        # a prompt prefilled into a contiguous cache [kv_heads, slots, dim] moved into pages
        _append("append_prompt_32761", 32761, 2, 128, 16, True),
        # a handful of interactive requests: the smallest attention call, latency counts
        _attend("decode_8_ctx1024", 8, 900, 1024, 1, 1, 12, 2, 128, 64, 3),
        # a mixed serving batch: lengths from a few tokens to 8192, small pages, q a slice of
        # the packed projection
        _attend("decode_64_ragged", 64, 1, 8191, 1, 1, 12, 2, 128, 16, 4, packed=True),
        # long contexts with sixteen query heads per kv head: the K/V stream
        _attend("decode_16_ctx32768", 16, 32700, 32767, 1, 1, 32, 2, 128, 64, 5),
        # four drafted tokens per request verified at once
        _attend("verify_32x4_ctx4096", 32, 3000, 4091, 4, 5, 12, 2, 128, 64, 6),
        # one 512-token chunk of a prompt on 3584 history slots
        _attend("chunk_512_on_3584", 1, 3584, 3584, 512, 512, 12, 2, 128, 64, 7),
        # prompts of odd lengths prefilled together, no history
        _attend("prompts_8_to_2000", 8, 0, 0, 700, 2000, 12, 2, 128, 32, 8),
        # a few requests behind one system prompt
        _attend("prefix_8_on_1024", 8, 1, 60, 1, 1, 12, 2, 128, 64, 9, prefix=1024),
        # many requests behind one long document
        _attend("prefix_128_on_16384", 128, 1, 500, 1, 1, 32, 2, 128, 64, 10, prefix=16384),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ((12, 2, 128), (32, 2, 128), (4, 2, 64), (16, 16, 64), (8, 4, 128), (32, 8, 64),
          (16, 4, 128))


def draw(rng):
    op = rng.choice(("plan", "append", "attend", "attend", "attend", "prefix"))
    page = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    if op == "plan":
        c = _plan("", _spread(rng, 1, 512), 0, _spread(rng, 1, 4096), 1,
                  rng.choice((1, 1, _spread(rng, 2, 400))), page, mix)
    elif op == "append":
        _, kv, dim = rng.choice(_HEADS)
        c = _append("", _spread(rng, 1, 32768 * 256 // (kv * dim)), kv, dim, page,
                    rng.random() < 0.5)
    else:
        heads, kv, dim = rng.choice(_HEADS)
        per_slot = kv * dim * 4
        most = (256 << 20) // per_slot         # slots over all sequences
        kind = rng.choice(("one", "one", "few", "many"))
        if op == "prefix":
            kind = rng.choice(("one", "one", "few"))
        if kind == "many":
            new_hi = _spread(rng, 20, 1500)
            B = _spread(rng, 1, max(1, 6000 // new_hi))
            hi = _spread(rng, 1, 4096)
            while B * new_hi * (hi + new_hi) * heads > 300e6:
                hi = hi // 2
                new_hi = max(20, new_hi * 3 // 4)
            new_lo = max(1, new_hi // 3)
        else:
            new_hi = 1 if kind == "one" else rng.randint(2, 9)
            new_lo = 1
            B = _spread(rng, 1, 200)
            hi = _spread(rng, 1, min(32768, max(2, most // B)))
        pre = 0
        if op == "prefix":
            pre = page * max(1, _spread(rng, 128, 16384) // page)
            hi = max(1, min(hi, 1024))
            while B * new_hi * (hi + pre) * heads > 60e6:
                B, hi, pre = B * 3 // 4, max(1, hi // 2), max(page, pre // 2 // page * page)
            B = max(2, B)
        c = _attend("", B, rng.randint(0, hi), hi, new_lo, new_hi, heads, kv, dim, page, mix,
                    prefix=pre, packed=rng.random() < 0.3)
    del c["name"]
    return c


def _lengths(c):
    """(history beyond the prefix, new tokens) of every sequence: the case's own."""
    rng = random.Random(c["mix"])
    return ([rng.randint(c["lo"], c["hi"]) for _ in range(c["B"])],
            [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])])


def work(c):
    if c["op"] == "plan":
        hist, new = _lengths(c)
        page, n, B = c["page"], sum(new), c["B"]
        taken = sum(-(-(h + t) // page) - -(-h // page) for h, t in zip(hist, new))
        # lengths and free pages read; starts, new table entries, slots and positions written
        return {"bytes": B * 16 + taken * 8 + (B + 1) * 8 + n * 16, "flops": n * 4}
    if c["op"] == "append":
        row = c["kv_heads"] * c["dim"] * 2
        return {"bytes": c["rows"] * (4 * row + 8), "flops": 0}
    hist, new = _lengths(c)
    heads, kv, dim, pre = c["heads"], c["kv_heads"], c["dim"], c["prefix"]
    slots = pre + sum(h + t for h, t in zip(hist, new))
    seen = sum(t * (pre + h) + t * (t + 1) // 2 for h, t in zip(hist, new))
    return {"bytes": slots * kv * dim * 4 + 2 * sum(new) * heads * dim * 2 +
            4 * (slots // c["page"]) + 16 * c["B"],
            "flops": 4 * dim * heads * seen}


# ---------------------------------------------------------------- inputs
def _block(heads, kv_heads, dim):
    """The library handle of these head counts (one per process, as a program keeps it)."""
    import decode_qwen2_block_gb300 as blk
    key = (heads, kv_heads, dim)
    if key not in _blocks:
        class Shape:
            hidden, n_heads, n_kv_heads, head_dim = heads * dim, heads, kv_heads, dim
            intermediate, has_qkv_bias, rms_eps, rope_theta = heads * dim, False, 1e-6, 1e4
        _blocks[key] = blk.Block(Shape, 1024)
    return _blocks[key]


def _pages(gen, n):
    return torch.randperm(n, generator=gen, device=_DEV).to(torch.int32)


def prepare(c, seed):
    gen = torch.Generator(_DEV)
    gen.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "append":
        n, kv, dim, page = c["rows"], c["kv_heads"], c["dim"], c["page"]
        n_pages = -(-n // page) + 3
        shape = (kv, n, dim) if c["head_major"] else (n, kv, dim)
        for name in ("k", "v"):
            t = torch.randn(shape, generator=gen, device=_DEV).half()
            s[name] = t.transpose(0, 1) if c["head_major"] else t
            s[name + "_pages"] = torch.zeros((n_pages, kv, page, dim), dtype=torch.float16,
                                             device=_DEV)
        r = torch.arange(n, device=_DEV)
        s["slots"] = _pages(gen, n_pages).long()[r // page] * page + r % page
        if own:
            s["block"] = _block(kv, kv, dim)
        return s

    hist, new = _lengths(c)
    page, pre, B = c["page"], c.get("prefix", 0), c["B"]
    lens = torch.tensor([pre + h for h in hist], dtype=torch.int64, device=_DEV)
    news = torch.tensor(new, dtype=torch.int64, device=_DEV)
    held = -(-lens // page)
    need = -(-(lens + news) // page)
    max_blocks = -(-(pre + c["hi"] + c["new_hi"]) // page)
    first = pre // page                        # table entries of the shared prefix
    col = torch.arange(max_blocks, device=_DEV)
    if c["op"] == "plan":
        total = int((need - held).sum())
        ids = _pages(gen, int(held.sum()) + total + 5)
        s["free"] = ids[:total + 5].contiguous()
        start = torch.cumsum(held, 0) - held + total + 5
        last = held
    else:
        ids = _pages(gen, first + int((need - first).sum()) + 2)
        start = torch.cumsum(need - first, 0) - (need - first)
        last = need
    at = torch.where(col < first, col, start[:, None] + col) if c["op"] != "plan" else \
        start[:, None] + col
    s["table"] = torch.where(col < last[:, None], ids[at.clamp(max=ids.numel() - 1)],
                             -1).to(torch.int32).contiguous()
    s["lens"], s["news"] = lens, news
    n = sum(new)
    s["row_start"] = torch.zeros(B + 1, dtype=torch.int64, device=_DEV)
    if c["op"] == "plan":
        s["slots"] = torch.empty(n, dtype=torch.int64, device=_DEV)
        s["pos"] = torch.empty(n, dtype=torch.int64, device=_DEV)
        s["used"] = torch.empty(1, dtype=torch.int64, device=_DEV)
        if own:
            s["block"] = _block(12, 2, 128)
        return s

    torch.cumsum(news, 0, out=s["row_start"][1:])
    heads, kv, dim = c["heads"], c["kv_heads"], c["dim"]
    width = (heads + 2 * kv if c["packed"] else heads) * dim
    q = torch.randn((n, width), generator=gen, device=_DEV).half()
    s["q"] = q[:, :heads * dim].unflatten(1, (heads, dim))
    for name in ("k_pages", "v_pages"):
        s[name] = torch.randn((ids.numel(), kv, page, dim), generator=gen, device=_DEV).half()
    s["prefix"] = ids[:first].contiguous() if pre else None
    s["max_new"], s["max_len"] = max(new), pre + max(h + t for h, t in zip(hist, new))
    s["out"] = torch.empty((n, heads, dim), dtype=torch.float16, device=_DEV)
    if own:
        b = s["block"] = _block(heads, kv, dim)
        s["batch"] = b.paged_batch(s["row_start"], lens, s["table"], n, page, ids.numel(),
                                   s["max_new"], s["max_len"], prefix_pages=s["prefix"])
        s["ws"] = torch.empty(b.attn_paged_workspace_bytes(n, B), dtype=torch.uint8, device=_DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_plan(s):
    page, lens, news = s["c"]["page"], s["lens"], s["news"]
    n = s["slots"].numel()
    ends = torch.cumsum(news, 0)
    starts = ends - news
    held = (lens + page - 1) // page
    need = (lens + news + page - 1) // page - held
    base = torch.cumsum(need, 0) - need
    table = s["table"]
    col = torch.arange(table.shape[1], device=table.device)
    k = col - held[:, None]
    fresh = (k >= 0) & (k < need[:, None])
    at = (base[:, None] + k).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], table)
    row = torch.arange(n, device=table.device)
    seq = torch.repeat_interleave(torch.arange(news.numel(), device=table.device), news,
                                  output_size=n)
    slot = lens[seq] + row - starts[seq]
    slots = table[seq, slot // page].long() * page + slot % page
    return {"table": table, "row_start": torch.cat((starts, ends[-1:])), "slots": slots,
            "pos": slot, "used": need.sum().reshape(1)}


def _plain_append(s):
    page = s["c"]["page"]
    where, off = s["slots"] // page, s["slots"] % page
    s["k_pages"][where, :, off] = s["k"]
    s["v_pages"][where, :, off] = s["v"]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    c = s["c"]
    heads, kv, dim, page, pre = c["heads"], c["kv_heads"], c["dim"], c["page"], c["prefix"]
    G, B, T, n = heads // kv, c["B"], s["max_new"], s["out"].shape[0]
    lens, news, dev = s["lens"], s["news"], s["q"].device
    seq = torch.repeat_interleave(torch.arange(B, device=dev), news, output_size=n)
    t = torch.arange(n, device=dev) - s["row_start"][seq]
    q = torch.zeros((B, T, heads, dim), device=dev)
    q[seq, t] = s["q"].float()
    q = q.view(B, T, kv, G, dim).permute(0, 2, 3, 1, 4).reshape(B, kv, G * T, dim)
    q = q / math.sqrt(dim)
    table = s["table"][:, pre // page:].long().clamp(min=0)      # each sequence's own pages
    k = s["k_pages"][table].float().transpose(1, 2).reshape(B, kv, -1, dim)
    v = s["v_pages"][table].float().transpose(1, 2).reshape(B, kv, -1, dim)
    slot = pre + torch.arange(k.shape[2], device=dev)
    last = (lens[:, None] + torch.arange(T, device=dev)).repeat(1, G)     # [B, G * T]
    score = q @ k.transpose(2, 3)
    score = score.masked_fill((slot > last[..., None])[:, None], -math.inf)
    if pre:
        pk = s["k_pages"][s["prefix"].long()].float().transpose(0, 1).reshape(kv, -1, dim)
        pv = s["v_pages"][s["prefix"].long()].float().transpose(0, 1).reshape(kv, -1, dim)
        qp = q.transpose(0, 1).reshape(kv, -1, dim)              # all rows of all sequences
        ps = (qp @ pk.transpose(1, 2)).view(kv, B, G * T, pre).transpose(0, 1)
        score = torch.cat((ps, score), -1)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    o = e[..., pre:] @ v
    if pre:
        ep = e[..., :pre].transpose(0, 1).reshape(kv, -1, pre)
        o = o + (ep @ pv).view(kv, B, G * T, dim).transpose(0, 1)
    o = o / e.sum(-1, keepdim=True)
    o = o.view(B, kv, G, T, dim).permute(0, 3, 1, 2, 4).reshape(B, T, heads, dim)
    return o[seq, t].half()


def run(s):
    c = s["c"]
    if own:
        b = s["block"]
        if c["op"] == "plan":
            b.page_plan(c["page"], s["lens"], s["news"], s["free"], s["table"], s["row_start"],
                        s["slots"], s["pos"], s["used"])
            return {"table": s["table"], "row_start": s["row_start"], "slots": s["slots"],
                    "pos": s["pos"], "used": s["used"]}
        if c["op"] == "append":
            b.page_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        b.attn_paged(s["batch"], s["q"], s["k_pages"], s["v_pages"], s["out"], s["ws"])
        return s["out"]
    if c["op"] == "plan":
        return _plain_plan(s)
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


# ---------------------------------------------------------------- in 64 bits
def _exact_plan(s):
    page = s["c"]["page"]
    lens, news, free = s["lens"].tolist(), s["news"].tolist(), s["free"].tolist()
    table = s["table"].tolist()
    starts, slots, pos, used = [0], [], [], 0
    for b, (have, more) in enumerate(zip(lens, news)):
        for i in range(-(-have // page), -(-(have + more) // page)):
            table[b][i] = free[used]
            used += 1
        for p in range(have, have + more):
            slots.append(table[b][p // page] * page + p % page)
            pos.append(p)
        starts.append(starts[-1] + more)
    whole = lambda x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    return {"table": whole(table).to(torch.int32), "row_start": whole(starts),
            "slots": whole(slots), "pos": whole(pos), "used": whole([used])}


def _exact_append(s):
    page = s["c"]["page"]
    got = {}
    for name, rows in (("k_pages", s["k"]), ("v_pages", s["v"])):
        flat = s[name].transpose(1, 2).contiguous().double()     # [pages, page, kv, dim]
        flat.view(-1, *flat.shape[2:]).index_copy_(0, s["slots"], rows.double())
        got[name] = flat.view(-1, page, *flat.shape[2:]).transpose(1, 2).contiguous()
    return got


def _exact_attend(s):
    """Sequence by sequence, head by head, from the softmax's definition."""
    c = s["c"]
    heads, kv, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (have, more) in enumerate(zip(s["lens"].tolist(), s["news"].tolist())):
        total = have + more
        pages = s["table"][b, :-(-total // page)].long()
        mine = lambda pool: pool[pages].transpose(0, 1).flatten(1, 2)[:, :total]  # noqa: E731
        k, v = mine(s["k_pages"]), mine(s["v_pages"])
        for h in range(heads):
            kh, vh = k[h // (heads // kv)].double(), v[h // (heads // kv)].double()
            z = s["q"][at:at + more, h].double() @ kh.T * dim ** -0.5
            row = torch.arange(more, device=z.device)[:, None]
            z = torch.where(torch.arange(total, device=z.device) <= have + row, z, -math.inf)
            out[at:at + more, h] = torch.softmax(z, -1) @ vh
        at += more
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "plan":
        return _exact_plan(s)
    if c["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s)
