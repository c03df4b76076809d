"""The operators of a paged K/V cache held in 8 bits: their plain forms, the
library's calls, and the cases both are measured on.

  append   K/V rows quantised into their pages by slot map, and read back as the
           attention will see them (``Block.page_append_kv8``, then
           ``Block.page_read_kv8`` of the same slots)
  read     slots of the cache back to fp16 rows, into a contiguous cache or packed
           rows (``Block.page_read_kv8``)
  attend   attention of a ragged batch over such caches: one new token per
           sequence, a few drafts, prompt chunks or whole prompts
           (``Block.attn_paged_kv8``)
  prefix   the same for a batch whose sequences share their first slots

A row (slot, kv head) of dim values is dim / 32 blocks of 32 columns.  With a the
greatest magnitude of a block, its scale s is the least E5M2 number with
127 s / 64 >= a, its codes are c = rint(64 x / s) (ties to even), stored as
c + 128 in a byte, and it stands for c s / 64.

With ``own`` false ``run`` is the plain form in elementary torch operations
(fp32, rounded once at the end); with ``own`` true it makes the library's calls.

Pools are codes uint8 [n_pages, kv_heads, page, dim] and scales float8_e5m2
[n_pages, kv_heads, page, dim / 32].  Row t of sequence b sits in slot
cache_lens[b] + t and sees slots [0, cache_lens[b] + t].
"""
import math
import random

import numpy as np
import torch

own = False

_DEV = "cuda"
_BLOCK = 32
_blocks = {}


# ---------------------------------------------------------------- cases
def _append(name, rows, kv_heads, dim, page, head_major):
    return {"name": name, "op": "append", "rows": rows, "kv_heads": kv_heads, "dim": dim,
            "page": page, "head_major": head_major}


def _read(name, rows, kv_heads, dim, page, head_major):
    return {"name": name, "op": "read", "rows": rows, "kv_heads": kv_heads, "dim": dim,
            "page": page, "head_major": head_major}


def _attend(name, B, lo, hi, new_lo, new_hi, heads, kv_heads, dim, page, mix, prefix=0,
            packed=False):
    return {"name": name, "op": "prefix" if prefix else "attend", "B": B, "lo": lo, "hi": hi,
            "new_lo": new_lo, "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "mix": mix, "prefix": prefix, "packed": packed}


def listed():
    return [
        # the K/V rows of one decode step of 64 requests: latency counts
        _append("append_step_64", 64, 2, 128, 64, False),
        # a prompt prefilled into a contiguous cache [kv_heads, slots, dim] moved into pages
        _append("append_prompt_32761", 32761, 2, 128, 16, True),
        # one request of odd length moved out to a contiguous cache
        _read("read_one_1031", 1031, 4, 128, 64, True),
        # many requests' slots moved out as packed rows
        _read("read_all_120007", 120007, 2, 128, 16, False),
        # a handful of interactive requests: the smallest attention call
        _attend("decode_8_ctx1024", 8, 900, 1024, 1, 1, 12, 2, 128, 64, 3),
        # a mixed serving batch: lengths from a few tokens to 12000, small pages, q a slice of
        # the packed projection
        _attend("decode_96_ragged", 96, 1, 12000, 1, 1, 12, 2, 128, 16, 4, packed=True),
        # contexts of 128 k tokens, sixteen query heads per kv head: the K/V stream
        _attend("decode_8_ctx131072", 8, 130900, 131071, 1, 1, 32, 2, 128, 64, 5),
        # small heads, one sequence's context beside another's, mid-sized pages
        _attend("decode_48_dim64", 48, 900, 6000, 1, 1, 32, 8, 64, 32, 11),
        # drafted tokens of every request verified at once
        _attend("verify_24x8_ctx6000", 24, 4000, 5990, 7, 8, 16, 4, 128, 64, 6),
        # one 1000-token chunk of a prompt behind 7000 slots
        _attend("chunk_1000_on_7000", 1, 7000, 7000, 1000, 1000, 12, 2, 128, 64, 7),
        # prompts of odd lengths prefilled together, no history
        _attend("prompts_12_to_1500", 12, 0, 0, 300, 1500, 12, 2, 128, 32, 8),
        # many requests behind one long document
        _attend("prefix_64_on_16384", 64, 1, 500, 1, 1, 32, 2, 128, 64, 10, prefix=16384),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ((12, 2, 128), (32, 2, 128), (4, 2, 64), (16, 16, 64), (8, 4, 128), (32, 8, 64),
          (16, 4, 128))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend", "attend", "prefix"))
    page = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    if op in ("append", "read"):
        _, kv, dim = rng.choice(_HEADS)
        most = 32768 * 256 if op == "append" else 120000 * 256
        make = _append if op == "append" else _read
        c = make("", _spread(rng, 1, most // (kv * dim)), kv, dim, page, rng.random() < 0.5)
    else:
        heads, kv, dim = rng.choice(_HEADS)
        most = (512 << 20) // (kv * dim * 2)   # slots over all sequences
        kind = rng.choice(("one", "one", "few", "many"))
        if op == "prefix":
            kind = rng.choice(("one", "one", "few"))
        if kind == "many":
            new_hi = _spread(rng, 20, 1500)
            B = _spread(rng, 1, max(1, 6000 // new_hi))
            hi = _spread(rng, 1, 7000)
            while B * new_hi * (hi + new_hi) * heads > 100e6:
                hi = hi // 2
                new_hi = max(20, new_hi * 3 // 4)
            new_lo = max(1, new_hi // 3)
        else:
            new_hi = 1 if kind == "one" else rng.randint(2, 9)
            new_lo = 1
            B = _spread(rng, 1, 200)
            hi = _spread(rng, 1, min(131071, max(2, most // B)))
            while B * new_hi * hi * heads > 100e6:
                hi = max(1, hi // 2)
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
    if c["op"] in ("append", "read"):
        n = c["rows"] * c["kv_heads"] * c["dim"] * 2       # values of K and V
        held = n + n // _BLOCK                             # their bytes in the cache
        # append: fp16 read, codes and scales written, fp16 written; read: without the first
        return {"bytes": held + 2 * n + (2 * n if c["op"] == "append" else 0) + 8 * c["rows"],
                "flops": 2 * n}
    hist, new = _lengths(c)
    heads, kv, dim, pre = c["heads"], c["kv_heads"], c["dim"], c["prefix"]
    slots = pre + sum(h + t for h, t in zip(hist, new))
    seen = sum(t * (pre + h) + t * (t + 1) // 2 for h, t in zip(hist, new))
    return {"bytes": slots * kv * 2 * (dim + dim // _BLOCK) + 2 * sum(new) * heads * dim * 2 +
            4 * (slots // c["page"]) + 16 * c["B"],
            "flops": 4 * dim * heads * seen}


# ---------------------------------------------------------------- the 8-bit form
def _quantise(x):
    """(codes uint8 [..., dim], scales float8_e5m2 [..., dim / 32]) of fp16 rows.  64 a / 127 and
    64 x / s are quotients of whole numbers of at most 17 bits: fp32's nearest is a border
    only where the quotient is one."""
    b = x.float().unflatten(-1, (-1, _BLOCK))
    need = b.abs().amax(-1) * 64 / 127
    near = need.to(torch.float8_e5m2)
    up = (near.float() < need).to(torch.uint8)
    scale = (near.view(torch.uint8) + up).view(torch.float8_e5m2)
    s = scale.float()[..., None]
    c = torch.round(b * 64 / torch.where(s > 0, s, 1.0)) + 128
    return c.to(torch.uint8).flatten(-2), scale


def _values(codes, scales):
    """What codes [..., dim] with scales [..., dim / 32] stand for, in fp32 (exact)."""
    s = scales.float()[..., None] / 64
    return ((codes.float() - 128).unflatten(-1, (-1, _BLOCK)) * s).flatten(-2)


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


def _gains(gen, kv, dim):
    """Rotated keys have columns that are larger than the others in every row."""
    return torch.exp(0.5 * torch.randn((kv, 1, dim), generator=gen, device=_DEV))


def _pool(gen, n_pages, kv, page, dim, gain):
    """Codes and scales of random pages, some pages at a time."""
    codes = torch.empty((n_pages, kv, page, dim), dtype=torch.uint8, device=_DEV)
    scales = torch.empty((n_pages, kv, page, dim // _BLOCK), dtype=torch.float8_e5m2, device=_DEV)
    some = max(1, (1 << 25) // (kv * page * dim))
    for i in range(0, n_pages, some):
        m = min(some, n_pages - i)
        x = torch.randn((m, kv, page, dim), generator=gen, device=_DEV) * gain
        codes[i:i + m], part = _quantise(x.half())
        scales[i:i + m].view(torch.uint8).copy_(part.view(torch.uint8))
    return codes, scales


def prepare(c, seed):
    gen = torch.Generator(_DEV)
    gen.manual_seed(seed)
    s = {"c": c}
    kv, dim, page = c["kv_heads"], c["dim"], c["page"]
    if c["op"] in ("append", "read"):
        n = c["rows"]
        n_pages = -(-n // page) + 3
        r = torch.arange(n, device=_DEV)
        s["slots"] = _pages(gen, n_pages).long()[r // page] * page + r % page
        shape = (kv, n, dim) if c["head_major"] else (n, kv, dim)
        for name in ("k", "v"):
            back = torch.empty(shape, dtype=torch.float16, device=_DEV)
            s[name + "_back"] = back.transpose(0, 1) if c["head_major"] else back
            gain = _gains(gen, kv, dim) if name == "k" else 1.0
            if c["op"] == "read":
                s[name + "_pages"], s[name + "_scales"] = _pool(gen, n_pages, kv, page, dim, gain)
                continue
            x = torch.randn((kv, n, dim), generator=gen, device=_DEV) * gain
            x = x.half()
            s[name] = x.transpose(0, 1) if c["head_major"] else x.transpose(0, 1).contiguous()
            s[name + "_pages"] = torch.zeros((n_pages, kv, page, dim), dtype=torch.uint8,
                                             device=_DEV)
            s[name + "_scales"] = torch.zeros((n_pages, kv, page, dim // _BLOCK),
                                              dtype=torch.uint8,
                                              device=_DEV).view(torch.float8_e5m2)
        if own:
            s["block"] = _block(kv, kv, dim)
        return s

    hist, new = _lengths(c)
    pre, B = c["prefix"], c["B"]
    lens = torch.tensor([pre + h for h in hist], dtype=torch.int64, device=_DEV)
    news = torch.tensor(new, dtype=torch.int64, device=_DEV)
    need = -(-(lens + news) // page)
    max_blocks = -(-(pre + c["hi"] + c["new_hi"]) // page)
    first = pre // page                        # table entries of the shared prefix
    col = torch.arange(max_blocks, device=_DEV)
    ids = _pages(gen, first + int((need - first).sum()) + 2)
    start = torch.cumsum(need - first, 0) - (need - first)
    at = torch.where(col < first, col, start[:, None] + col)
    s["table"] = torch.where(col < need[:, None], ids[at.clamp(max=ids.numel() - 1)],
                             -1).to(torch.int32).contiguous()
    s["lens"], s["news"] = lens, news
    n = sum(new)
    s["row_start"] = torch.zeros(B + 1, dtype=torch.int64, device=_DEV)
    torch.cumsum(news, 0, out=s["row_start"][1:])
    heads = c["heads"]
    width = (heads + 2 * kv if c["packed"] else heads) * dim
    q = torch.randn((n, width), generator=gen, device=_DEV).half()
    s["q"] = q[:, :heads * dim].unflatten(1, (heads, dim))
    for name in ("k", "v"):
        gain = _gains(gen, kv, dim) if name == "k" else 1.0
        s[name + "_pages"], s[name + "_scales"] = _pool(gen, ids.numel(), kv, page, dim, gain)
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
def _plain_append(s, name):
    page = s["c"]["page"]
    where, off = s["slots"] // page, s["slots"] % page
    codes, scales = _quantise(s[name])
    s[name + "_pages"][where, :, off] = codes
    s[name + "_scales"].view(torch.uint8)[where, :, off] = scales.view(torch.uint8)


def _plain_read(s, name):
    page = s["c"]["page"]
    where, off = s["slots"] // page, s["slots"] % page
    scales = s[name + "_scales"].view(torch.uint8)[where, :, off].view(torch.float8_e5m2)
    return _values(s[name + "_pages"][where, :, off], scales).half()


def _pages_of(s, name, table):
    """The values of the pages of `table` [..., blocks]: fp32 [..., blocks, kv, page, dim]."""
    scales = s[name + "_scales"].view(torch.uint8)[table].view(torch.float8_e5m2)
    return _values(s[name + "_pages"][table], scales)


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
    k = _pages_of(s, "k", table).transpose(1, 2).reshape(B, kv, -1, dim)
    v = _pages_of(s, "v", table).transpose(1, 2).reshape(B, kv, -1, dim)
    slot = pre + torch.arange(k.shape[2], device=dev)
    last = (lens[:, None] + torch.arange(T, device=dev)).repeat(1, G)     # [B, G * T]
    score = q @ k.transpose(2, 3)
    score = score.masked_fill((slot > last[..., None])[:, None], -math.inf)
    if pre:
        pk = _pages_of(s, "k", s["prefix"].long()).transpose(0, 1).reshape(kv, -1, dim)
        pv = _pages_of(s, "v", s["prefix"].long()).transpose(0, 1).reshape(kv, -1, dim)
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
    op = s["c"]["op"]
    if own:
        b = s["block"]
        pools = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if op in ("append", "read"):
            if op == "append":
                b.page_append_kv8(s["k"], s["v"], s["slots"], *pools)
            b.page_read_kv8(s["slots"], *pools, s["k_back"], s["v_back"])
            return {"k": s["k_back"], "v": s["v_back"]}
        b.attn_paged_kv8(s["batch"], s["q"], *pools, s["out"], s["ws"])
        return s["out"]
    if op in ("append", "read"):
        if op == "append":
            _plain_append(s, "k")
            _plain_append(s, "v")
        return {"k": _plain_read(s, "k"), "v": _plain_read(s, "v")}
    return _plain_attend(s)


# ---------------------------------------------------------------- in 64 bits
def _exact_rows(x):
    """Rows [n, kv, dim] as the cache holds them, from the definition, in numpy's 64 bits."""
    x = x.cpu().numpy().astype(np.float64).reshape(x.shape[0], x.shape[1], -1, _BLOCK)
    need = np.abs(x).max(-1, keepdims=True) * 64 / 127
    _, e = np.frexp(need)                      # need in [2^(e - 1), 2^e): E5M2 steps 2^(e - 3)
    step = np.ldexp(1.0, np.maximum(e - 3, -16))
    s = np.ceil(need / step) * step
    c = np.rint(x * 64 / np.where(s > 0, s, 1.0))
    return torch.from_numpy((c * s / 64).reshape(*x.shape[:2], -1))


def _exact_pages(s, name, pages):
    """Pages of the pool in 64 bits."""
    codes = s[name + "_pages"][pages].double().unflatten(-1, (-1, _BLOCK)) - 128
    scales = s[name + "_scales"].view(torch.uint8)[pages].view(torch.float8_e5m2).double()
    return (codes * (scales[..., None] / 64)).flatten(-2)


def _exact_attend(s):
    """Sequence by sequence, head by head, from the softmax's definition."""
    c = s["c"]
    heads, kv, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (have, more) in enumerate(zip(s["lens"].tolist(), s["news"].tolist())):
        total = have + more
        pages = s["table"][b, :-(-total // page)].long()
        k, v = (_exact_pages(s, name, pages).transpose(0, 1).flatten(1, 2)[:, :total]
                for name in ("k", "v"))
        for h in range(heads):
            z = s["q"][at:at + more, h].double() @ k[h // (heads // kv)].T * dim ** -0.5
            row = torch.arange(more, device=z.device)[:, None]
            z = torch.where(torch.arange(total, device=z.device) <= have + row, z, -math.inf)
            out[at:at + more, h] = torch.softmax(z, -1) @ v[h // (heads // kv)]
        at += more
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        return {"k": _exact_rows(s["k"]), "v": _exact_rows(s["v"])}
    if c["op"] == "read":
        page = c["page"]
        where, off = s["slots"] // page, s["slots"] % page
        got = {}
        for name in ("k", "v"):
            whole = _exact_pages(s, name, slice(None))
            got[name] = whole[where, :, off]
        return got
    return _exact_attend(s)
