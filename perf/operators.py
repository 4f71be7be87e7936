"""The paged 4-bit cache's operators as a serving program calls them: cases, inputs, plain forms and exact values.

  append   quantise new keys and values into the pages of their sequences, and read them back as the cache holds them
  attend   attention of each sequence's newest tokens over its pages (single tokens, a few, a prompt's chunk)
  sparse   choose each sequence's pages by a cheap score, and attend to the chosen ones alone
  fork     a beam step: children take their parents' pages, the parents go, each child gets room for one more token
  compact  sequences end, the pages of the others move down, new sequences take pages

A page of one layer and KV head is P tokens in blocks of b = min(P, 64):
  key codes   [b][d / 2]              channel 2j in the low half of byte j, 2j + 1 in the high half
  key scales  [b][d / 16]             one e4m3 scale for 16 channels
  value codes [b / 8][d / 16][4][16]  8 tokens, 16 channels, pair of tokens, channel: the even token in the low half
  value scales[b / 8][d / 16][4][2]   the same order, the two tokens of a pair side by side
A value is 2^exp * scale * code, its code one of 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign (e2m1).  The summary of a page
holds, for each channel, the largest and the smallest key among its tokens as whole numbers of 8 bits (rounded up and
down) times 2^e: [d] largest, [d] smallest, int32 e, 12 bytes of nothing.
"""
import math
import random

import torch

own = False  # the framework's calls in place of the plain forms

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BOUNDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between the magnitudes; a tie goes to the even code


# ---- cases -----------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(op=op, dtype="bf16", d=128, hkv=8, g=4, page=64, layers=1, rows=1, lo=1, hi=1, new_lo=1, new_hi=1,
             empty=0, k_exp=0, v_exp=-2, salt=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's next token enters the cache: nothing but latency
        _case("append 1x1", "append", lo=301, hi=301),
        # a full batch's decode step at ragged lengths, two layers in the pool
        _case("append 64x1 f16 p16", "append", dtype="f16", page=16, layers=2, rows=64, lo=1, hi=2048, salt=2),
        # prompts of a batch enter the cache behind what their conversations hold
        _case("append 16 prompts", "append", rows=16, lo=4096, hi=9000, new_lo=2048, new_hi=8192, salt=3),
        # one user's short conversation, head dim 64, one query head for each KV head
        _case("attend 1x1 s500 d64", "attend", dtype="f16", d=64, g=1, page=16, lo=500, hi=500, salt=4),
        # the decode step of a batch of 16 at 8192 tokens, 32 query and 8 KV heads
        _case("attend 16x1 s8192", "attend", rows=16, lo=8192, hi=8192, salt=5),
        # ragged decode with a padded batch, 8 query heads for each KV head
        _case("attend 40x1 ragged g8", "attend", g=8, page=32, rows=40, lo=3, hi=16384, empty=3, salt=6),
        # a proposal of a few tokens is checked over long conversations
        _case("attend 8x4 s32768 p128", "attend", page=128, rows=8, lo=30001, hi=32768, new_lo=3, new_hi=4, salt=7),
        # a prompt's chunk over what came before it
        _case("attend 1x2048 s16384", "attend", lo=16384, hi=16384, new_lo=2048, new_hi=2048, salt=8),
        # one long conversation: 64 of 2048 pages
        _case("sparse 1x1 s131072 k64", "sparse", lo=131072, hi=131072, keep=64, salt=9),
        # a batch at 32768 tokens: 48 of 512 pages and shorter ones
        _case("sparse 16x1 s32768 k48", "sparse", dtype="f16", rows=16, lo=1500, hi=32768, keep=48, salt=10),
        # a beam search over 16 requests of 4 beams, 32 layers
        _case("fork 64 beams 32 layers", "fork", layers=32, rows=64, lo=90, hi=500, salt=11),
        # half of a batch ends, the other half's pages move down, 8 layers
        _case("compact 32 rows 8 layers", "compact", layers=8, rows=32, lo=700, hi=4000, salt=12),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["append", "attend", "attend", "sparse", "fork", "compact"])
        kw = dict(dtype=rng.choice(["bf16", "f16"]), d=rng.choice([64, 128, 128]), hkv=rng.choice([1, 2, 4, 8]),
                  g=rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), page=rng.choice([16, 32, 64, 128]), salt=rng.randrange(1 << 20),
                  k_exp=rng.choice([0, 0, 2, -3]), v_exp=rng.choice([0, -2, -5]))
        if op == "append":
            kw.update(rows=size(1, 64), hi=size(1, 9000), new_hi=size(1, 8192), layers=rng.choice([1, 2]))
        elif op == "attend":
            new = rng.choice([1, 1, size(2, 16), size(17, 2048)])
            kw.update(rows=size(1, 64), hi=size(1, 32768), new_hi=new, new_lo=1 if rng.random() < 0.5 else new,
                      empty=rng.choice([0, 0, 1]), layers=rng.choice([1, 1, 2]))
        elif op == "sparse":
            kw.update(rows=size(1, 32), hi=size(64, 131072), keep=size(3, 128))
        elif op == "fork":
            kw.update(rows=rng.choice([4 * size(1, 32), size(1, 128)]), hi=size(2, 4000), layers=size(1, 32))
        else:
            kw.update(rows=2 * size(1, 24), hi=size(2, 6000), layers=size(1, 16))
        kw["lo"] = max(1, int(kw["hi"] * rng.choice([0.02, 0.5, 1.0])))
        if op == "append":
            kw["new_lo"] = max(1, int(kw["new_hi"] * rng.choice([0.05, 1.0])))
        c = _case("", op, **kw)
        if _cost(c) <= most and _held(c) <= 40e9:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280)  # this card's flops for each byte


def _held(c):
    """Bytes that the plain form keeps at once, about."""
    lens, new, _ = _lengths(c)
    most = max(lens)
    if c["op"] in ("fork", "compact"):
        return _pool_pages(c) * c["layers"] * c["hkv"] * (_page_bytes(c) + 2 * c["d"] + 16) * 4
    if c["op"] == "append":
        return sum(new) * c["hkv"] * c["d"] * 100
    return len(lens) * most * c["hkv"] * c["d"] * 40 + len(lens) * max(new) * c["hkv"] * c["g"] * most * 12


def _lengths(c):
    """Each row's length with its new tokens, its new tokens, and (fork) its parent."""
    rng = random.Random(c["salt"] * 7 + 1)
    n = c["rows"] // 2 if c["op"] == "compact" else c["rows"]
    lens = [rng.randint(c["lo"], c["hi"]) for _ in range(n)]
    if n > 2:
        lens[0], lens[n // 2] = c["hi"], c["lo"]
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(n)]
    if c["op"] == "append":
        lens = [a + b for a, b in zip(lens, new)]
    new = [min(a, b) for a, b in zip(lens, new)]
    if c["empty"] and n > c["empty"]:  # rows of a padded batch: one query token and nothing in the cache
        lens[-c["empty"]:], new[-c["empty"]:] = [0] * c["empty"], [1] * c["empty"]
    if c["op"] == "compact":
        lens, new = lens + lens, new + new
    beams = 4 if n % 4 == 0 else 1
    parents = [i // beams * beams + rng.randrange(beams) for i in range(len(lens))]
    if c["op"] == "fork":
        lens = [lens[i // beams * beams] for i in range(n)]
    return lens, new, parents


def _page_bytes(c):
    return c["page"] * c["d"] * 9 // 8


def _pages(c, n):
    return -(-n // c["page"])


def _per_row(c):
    lens, _, _ = _lengths(c)
    return max(1, _pages(c, max(lens) + 1))


def _pool_pages(c):
    lens, _, _ = _lengths(c)
    n = sum(_pages(c, x) for x in lens)
    return n + 3 if c["op"] != "fork" else 2 * n + 2 * len(lens) + 3


def work(c):
    lens, new, parents = _lengths(c)
    d, hkv, g, tok = c["d"], c["hkv"], c["g"], c["hkv"] * c["d"] * 9 // 8  # bytes of a token's keys and values
    summary = hkv * (2 * d + 4)
    n = sum(new)
    if c["op"] == "append":
        touched = sum(_pages(c, x) - (x - y) // c["page"] for x, y in zip(lens, new))
        before = sum((x - y) % c["page"] for x, y in zip(lens, new))
        return {"bytes": 2 * 2 * n * hkv * d * 2 + 2 * n * tok + before * tok // 2 + touched * summary,
                "flops": 12 * n * hkv * d}
    if c["op"] == "attend":
        pairs = sum(max(0, y * x - y * (y - 1) // 2) for x, y in zip(lens, new))
        return {"bytes": 2 * n * hkv * g * d * 2 + n * hkv * g * 4 + sum(lens) * tok + 4 * sum(_pages(c, x) for x in lens),
                "flops": 4 * pairs * hkv * g * d}
    if c["op"] == "sparse":
        seen = [min(x, c["keep"] * c["page"]) for x in lens]
        every = sum(_pages(c, x) for x in lens)
        return {"bytes": 2 * n * hkv * g * d * 2 + every * (summary + 4) + sum(seen) * tok + 4 * hkv * c["keep"] * n,
                "flops": 4 * sum(seen) * hkv * g * d + 4 * every * hkv * d}
    if c["op"] == "fork":
        copies = len(lens) - len(set(parents))
        part = [x % c["page"] for x in lens]
        moved = c["layers"] * (copies * summary + int(copies * sum(part) / len(part) * tok))
        return {"bytes": 2 * moved + 12 * sum(_pages(c, x) + 1 for x in lens), "flops": 0}
    half = sum(_pages(c, x) for x in lens[: len(lens) // 2])
    return {"bytes": 2 * c["layers"] * half * (hkv * _page_bytes(c) + summary) + 32 * half, "flops": 0}


# ---- the page format, in torch -----------------------------------------------------------------------------------
def _quantise(x, exp):
    """x [..., d] in 32 bits -> codes [..., d], scales [..., d / 16] (e4m3)."""
    b = x.unflatten(-1, (-1, 16))
    top = b.abs().amax(-1)
    s = (top / torch.full_like(top, 6.0) * 2.0 ** -exp).clamp(max=448.0).to(torch.float8_e4m3fn)
    S = s.float().unsqueeze(-1) * 2.0 ** exp
    a = b.abs()
    code = ((a > BOUNDS[0] * S).byte() + (a >= BOUNDS[1] * S).byte() + (a > BOUNDS[2] * S).byte() + (a >= BOUNDS[3] * S).byte()
            + (a > BOUNDS[4] * S).byte() + (a >= BOUNDS[5] * S).byte() + (a > BOUNDS[6] * S).byte())
    code = code * (S > 0) + 8 * torch.signbit(b).byte()
    return code.flatten(-2), s


def _pack(kc, ks, vc, vs):
    """codes [..., P, d] and scales [..., P, d / 16] of a page -> its bytes."""
    P, d = kc.shape[-2:]
    b = min(P, 64)
    lead = kc.shape[:-2] + (P // b,)
    kb = (kc[..., 0::2] | kc[..., 1::2] << 4).reshape(*lead, -1)
    v = vc.reshape(*lead, b // 8, 4, 2, d // 16, 16)
    vb = (v[..., 0, :, :] | v[..., 1, :, :] << 4).transpose(-2, -3).reshape(*lead, -1)
    s = vs.view(torch.uint8).reshape(*lead, b // 8, 4, 2, d // 16)
    sb = s.movedim(-1, -3).reshape(*lead, -1)
    return torch.cat([kb, ks.view(torch.uint8).reshape(*lead, -1), vb, sb], -1).flatten(-2)


def _codes(raw, P, d):
    """A page's bytes [..., PB] -> key codes, key scales, value codes, value scales, as _pack takes them."""
    b = min(P, 64)
    r = raw.unflatten(-1, (P // b, -1))
    kb, ks, vb, vs = r.split([b * d // 2, b * d // 16, b * d // 2, b * d // 16], -1)
    kc = torch.stack([kb & 15, kb >> 4], -1).flatten(-2).unflatten(-1, (b, d)).flatten(-3, -2)
    v = vb.unflatten(-1, (b // 8, d // 16, 4, 16)).transpose(-2, -3)
    vc = torch.stack([v & 15, v >> 4], -3).flatten(-5, -3).flatten(-2).flatten(-3, -2)
    s = vs.unflatten(-1, (b // 8, d // 16, 4, 2)).movedim(-3, -1).flatten(-4, -2).flatten(-3, -2)
    return kc, ks.unflatten(-1, (b, -1)).flatten(-3, -2).contiguous().view(torch.float8_e4m3fn), vc, s.contiguous().view(torch.float8_e4m3fn)


def _table(device):
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([m, -m])


def _values(code, scale, exp):
    x = _table(code.device)[code.long()].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)
    return x.flatten(-2) * 2.0 ** exp


def _summary(x, count):
    """Largest and smallest key of each channel over the first `count` tokens of x [..., P, d] -> the summary's bytes."""
    inside = (torch.arange(x.shape[-2], device=x.device) < count.unsqueeze(-1)).unsqueeze(-1)
    top = torch.where(inside, x, -math.inf).amax(-2)
    low = torch.where(inside, x, math.inf).amin(-2)
    m = torch.maximum(top.abs(), low.abs()).amax(-1)
    e = torch.where(m > 0, torch.frexp(m).exponent - 7, 0).int()
    unit = torch.ldexp(torch.ones_like(m), -e).unsqueeze(-1)
    whole = torch.cat([torch.ceil(top * unit), torch.floor(low * unit)], -1).to(torch.int8).view(torch.uint8)
    tail = torch.cat([e.unsqueeze(-1), e.new_zeros(e.shape + (3,))], -1).view(torch.uint8)
    return torch.cat([whole, tail], -1)


# ---- inputs --------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed * 977 + 13)
    lens, new, parents = _lengths(c)
    R, P, d, hkv, L = len(lens), c["page"], c["d"], c["hkv"], c["layers"]
    M, N = _per_row(c), _pool_pages(c)
    held = [x - y if c["op"] == "append" else x for x, y in zip(lens, new)]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # keys with a mean of their own in every channel and a few channels ten times as large, as projections give them
    mean, wide = normal(hkv, 1, d) * math.sqrt(2.0), torch.ones(hkv, 1, d, device=dev)
    wide.view(-1)[torch.randperm(hkv * d, generator=gen, device=dev)[: max(1, hkv * d // 100)]] = 10.0

    s = {"case": c, "lens": lens, "new": new, "layer": L - 1, "max_new": max(new)}
    pages = torch.zeros(L, N, hkv, _page_bytes(c), dtype=torch.uint8, device=dev)
    summary = torch.zeros(L, N, hkv, 2 * d + 16, dtype=torch.uint8, device=dev)
    if c["op"] in ("fork", "compact"):  # what these pages hold is of no account to them
        pages.copy_(torch.randint(0, 256, pages.shape, generator=gen, device=dev, dtype=torch.uint8))
        summary.copy_(torch.randint(0, 256, summary.shape, generator=gen, device=dev, dtype=torch.uint8))
        order = torch.arange(N, device=dev)
    else:
        order = torch.randperm(N, generator=gen, device=dev)
    # each row's pages, in the pool's order or in a random one
    table = torch.full((2 * R if c["op"] == "fork" else R, M), -1, dtype=torch.int32, device=dev)
    refs = torch.zeros(N, dtype=torch.int32, device=dev)
    count = [_pages(c, x) for x in lens]  # append: room for the new tokens is there
    fill = [i for i, n in enumerate(count) for _ in range(n)]
    place = [j for n in count for j in range(n)]
    fill, place = torch.tensor(fill, device=dev), torch.tensor(place, device=dev)
    total = sum(count)
    table[fill, place] = order[:total].int()
    refs[order[:total]] = 1
    full = torch.zeros(N, dtype=torch.int64, device=dev)
    full[order[:total]] = (torch.tensor(held, device=dev)[fill] - place * P).clamp(0, P)
    if c["op"] not in ("fork", "compact"):
        for at in range(0, N, 256):  # a part of the pool at a time
            n = min(256, N - at)
            k = (normal(n, hkv, P, d) + mean) * wide
            v = normal(n, hkv, P, d) * 2.0 ** (c["v_exp"] + 2)
            kc, ks = _quantise(k, c["k_exp"])
            pages[L - 1, at:at + n] = _pack(kc, ks, *_quantise(v, c["v_exp"]))
            cnt = full[at:at + n].clamp(min=1).unsqueeze(-1).expand(n, hkv)
            summary[L - 1, at:at + n] = _summary(_values(kc, ks, 0), cnt)
    size = torch.tensor(lens + [0] * (table.shape[0] - R), dtype=torch.int32, device=dev)
    s.update(pages=pages, summary=summary, table=table, seq_len=size, refs=refs)
    dt = DTYPES[c["dtype"]]
    n = sum(new)
    one = max(new) == 1 and min(new) == 1
    s["cu"] = None if one else torch.tensor([sum(new[:i]) for i in range(R + 1)], dtype=torch.int32, device=dev)
    s["row"] = torch.tensor([i for i, y in enumerate(new) for _ in range(y)], device=dev)
    s["pos"] = torch.tensor([x - y + t for x, y in zip(lens, new) for t in range(y)], device=dev)
    s["turn"] = torch.tensor([t for y in new for t in range(y)], device=dev)
    if c["op"] == "append":
        s["k"] = ((normal(n, hkv, d) + mean.view(hkv, d)) * wide.view(hkv, d)).to(dt)
        s["v"] = (normal(n, hkv, d) * 2.0 ** (c["v_exp"] + 2)).to(dt)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        first = [(x - y) // P for x, y in zip(lens, new)]
        touched = [(i, j) for i, x in enumerate(lens) for j in range(first[i], _pages(c, x))]
        s["touched"] = torch.tensor(touched, device=dev)
        begin = [0]
        for i in range(R):
            begin.append(begin[-1] + _pages(c, lens[i]) - first[i])
        s["slot"] = torch.tensor(begin[:-1], device=dev)[s["row"]] + s["pos"] // P - torch.tensor(first, device=dev)[s["row"]]
    elif c["op"] in ("attend", "sparse"):
        s["q"] = normal(n, hkv * c["g"], d).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, hkv * c["g"], dtype=torch.float32, device=dev)
        s["sel"] = torch.empty(R, hkv, c.get("keep", 1), dtype=torch.int32, device=dev)
    elif c["op"] == "fork":
        i32 = dict(dtype=torch.int32, device=dev)
        s["sides"] = [torch.arange(R, **i32), torch.arange(R, 2 * R, **i32)]
        s["parent"] = torch.tensor(parents, **i32)
        s["sources"] = [s["parent"], s["parent"] + R]
        s["longer"], s["none"] = torch.tensor([x + 1 for x in lens], **i32), torch.zeros(R, **i32)
        s["back"] = torch.tensor(lens, **i32)
        s["at"] = 0
    else:
        i32 = dict(dtype=torch.int32, device=dev)
        s["sides"] = [torch.arange(0, R // 2, **i32), torch.arange(R // 2, R, **i32)]
        s["back"], s["none"] = torch.tensor(lens[: R // 2], **i32), torch.zeros(R // 2, **i32)
        s["at"] = 0
    return s


# ---- the framework's calls -------------------------------------------------------------------------------------------
def _pool(s):
    """The handle that a program keeps over its buffers."""
    if "pool" not in s:
        from quantized_decode_attention_gb300 import PagePool, make_pages_config
        c = s["case"]
        cfg = make_pages_config(n_layers=c["layers"], n_pages=s["pages"].shape[1], page_size=c["page"], n_kv_heads=c["hkv"],
                                n_q_heads=c["hkv"] * c["g"], head_dim=c["d"], max_seqs=s["table"].shape[0],
                                max_pages_per_seq=s["table"].shape[1], dtype=c["dtype"], k_exp=c["k_exp"], v_exp=c["v_exp"])
        s["pool"] = PagePool(cfg, pages=s["pages"], summary=s["summary"], table=s["table"], seq_len=s["seq_len"], refs=s["refs"])
    return s["pool"]


# ---- the plain forms ---------------------------------------------------------------------------------------------------
def _append(s):
    c, layer = s["case"], s["layer"]
    P, d = c["page"], c["d"]
    row, page = s["touched"][:, 0], s["touched"][:, 1]
    ids = s["table"][row, page].long()
    old = _codes(s["pages"][layer, ids], P, d)
    now = [x.clone() for x in old]
    inside = s["pos"] % P
    for_k, for_v = _quantise(s["k"].float(), c["k_exp"]), _quantise(s["v"].float(), c["v_exp"])
    now[0][s["slot"], :, inside], now[2][s["slot"], :, inside] = for_k[0], for_v[0]
    now[1].view(torch.uint8)[s["slot"], :, inside] = for_k[1].view(torch.uint8)
    now[3].view(torch.uint8)[s["slot"], :, inside] = for_v[1].view(torch.uint8)
    s["pages"][layer, ids] = _pack(*now)
    count = (s["seq_len"][row] - page * P).clamp(max=P)
    s["summary"][layer, ids] = _summary(_values(now[0], now[1], 0), count.unsqueeze(-1).expand(-1, c["hkv"]))
    kc, ks, vc, vs = _codes(s["pages"][layer, ids], P, d)
    dt = DTYPES[c["dtype"]]
    k = _values(kc, ks, c["k_exp"])[s["slot"], :, inside]
    v = _values(vc, vs, c["v_exp"])[s["slot"], :, inside]
    return k.to(dt), v.to(dt)


def _attend(s, sel=None):
    """Softmax attention in 32 bits of each row's newest tokens, over its pages or the chosen ones."""
    c = s["case"]
    P, hkv, g, d = c["page"], c["hkv"], c["g"], c["d"]
    table = s["table"].long()
    R, M = table.shape
    kc, ks, vc, vs = _codes(s["pages"][s["layer"]][table.clamp(min=0)], P, d)
    k, v = _values(kc, ks, c["k_exp"]), _values(vc, vs, c["v_exp"])  # [R, M, hkv, P, d]
    k, v = k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)  # [R, hkv, S, d]
    T, S = s["max_new"], M * P
    q = torch.zeros(R, T, hkv, g, d, device=k.device)
    q[s["row"], s["turn"]] = s["q"].float().unflatten(1, (hkv, g))
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, hkv, T * g, d]
    score = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    last = torch.full((R, T), -1, device=k.device)
    last[s["row"], s["turn"]] = s["pos"]
    ok = torch.arange(S, device=k.device) <= last.unsqueeze(-1)  # [R, T, S]
    ok = ok.unsqueeze(1).expand(R, hkv, T, S)
    if sel is not None:
        some = torch.zeros(R, hkv, M + 1, dtype=torch.bool, device=k.device)
        some.scatter_(2, torch.where(sel < 0, M, sel).long(), True)
        ok = ok & some[..., :M].repeat_interleave(P, -1).unsqueeze(2)
    score = score.masked_fill_(~ok.repeat_interleave(g, 2), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out, lse = (x.unflatten(2, (T, g)).transpose(1, 2)[s["row"], s["turn"]].flatten(1, 2) for x in (out, lse))
    return out.to(DTYPES[c["dtype"]]), lse


def _choose(s):
    """The pages that each KV head's query heads are thought to want most, ascending, then -1."""
    c = s["case"]
    hkv, g, d, keep = c["hkv"], c["g"], c["d"], c["keep"]
    R, M = s["table"].shape
    q = s["q"].double().unflatten(1, (hkv, g))
    high, low = q.clamp(min=0).sum(2).float(), q.clamp(max=0).sum(2).float()  # [R, hkv, d]
    top = torch.maximum(high, -low).amax(-1, keepdim=True)
    inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, 0.0)
    high, low = torch.round(high * inv), torch.round(low * inv)
    raw = s["summary"][s["layer"]][s["table"].long().clamp(min=0)].transpose(1, 2)  # [R, hkv, M, bytes]
    most, least = raw[..., :d].view(torch.int8).float(), raw[..., d:2 * d].view(torch.int8).float()
    e = raw[..., 2 * d:2 * d + 4].contiguous().view(torch.int32).squeeze(-1)
    score = torch.ldexp((most * high.unsqueeze(2) + least * low.unsqueeze(2)).sum(-1), e)  # whole numbers below 2^24: exact
    pages = ((s["seq_len"] + c["page"] - 1) // c["page"]).view(R, 1, 1)
    j = torch.arange(M, device=raw.device)
    score = torch.where((j < 1) | (j == pages - 1), math.inf, score)
    score = torch.where(j < pages, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < pages, best, M).sort(-1).values
    best = torch.where(best < M, best, -1).int()
    return torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=-1)


def _fork(s, src, dst):
    t = s["table"][src.long()]
    s["table"][dst.long()] = t
    s["seq_len"][dst.long()] = s["seq_len"][src.long()]
    s["refs"] += torch.bincount(t[t >= 0].long(), minlength=s["refs"].shape[0]).int()


def _resize(s, rows, size):
    """Give back the pages behind the new length; a shared last page that is written next is copied, all but its last
    writer's when nobody else holds it; then each row in turn takes the lowest free pages."""
    P = s["case"]["page"]
    table, refs, rows = s["table"], s["refs"], rows.long()
    before, j = s["seq_len"][rows], torch.arange(table.shape[1], device=table.device)
    had, has = (before + P - 1) // P, (size + P - 1) // P
    t = table[rows]
    drop = (j >= has.unsqueeze(1)) & (t >= 0)
    refs -= torch.bincount(t[drop].long(), minlength=refs.shape[0]).int()
    t = torch.where(drop, -1, t)
    grows = (size > before) & (before % P != 0)
    at = (before // P).long().clamp(max=table.shape[1] - 1)
    page = torch.where(grows, t.gather(1, at.unsqueeze(1)).squeeze(1), -1)
    i = torch.arange(len(rows), device=table.device)
    earlier = ((page.unsqueeze(0) == page.unsqueeze(1)) & grows & (i.unsqueeze(0) < i.unsqueeze(1))).sum(1)
    copy = grows & (refs[page.long().clamp(min=0)] - earlier > 1)
    need = copy.int() + (has - had).clamp(min=0)
    end = need.cumsum(0)
    free = (refs == 0).nonzero().squeeze(1).int()
    first = (end - need).unsqueeze(1)
    fresh = free[torch.where(copy, first.squeeze(1), 0).long()]
    source = page[copy].long()
    s["pages"][:, fresh[copy].long()] = s["pages"][:, source]
    s["summary"][:, fresh[copy].long()] = s["summary"][:, source]
    refs -= torch.bincount(source, minlength=refs.shape[0]).int()
    t = torch.where(copy.unsqueeze(1) & (j == at.unsqueeze(1)), fresh.unsqueeze(1), t)
    add = (j >= had.unsqueeze(1)) & (j < has.unsqueeze(1))
    k = first + copy.unsqueeze(1) + j - had.unsqueeze(1)
    t = torch.where(add, free[torch.where(add, k, 0).long()], t)
    refs[free[: int(end[-1])].long()] = 1
    table[rows] = t
    s["seq_len"][rows] = size


def _compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n = int(live.sum())
    src = live[n:].nonzero().squeeze(1) + n
    dst = (~live[:n]).nonzero().squeeze(1)
    s["pages"][:, dst], s["summary"][:, dst] = s["pages"][:, src], s["summary"][:, src]
    to = torch.arange(len(refs), device=refs.device, dtype=torch.int32)
    to[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], -1))


def run(s):
    op = s["case"]["op"]
    if op == "append":
        if own:
            p = _pool(s)
            p.append(s["layer"], s["k"], s["v"], cu=s["cu"], max_new=s["max_new"])
            p.read(s["layer"], s["k_out"], s["v_out"], cu=s["cu"], max_new=s["max_new"])
            k, v = s["k_out"], s["v_out"]
        else:
            k, v = _append(s)
        return {"k": k, "v": v, "pages": s["pages"].view(torch.int32), "summary": s["summary"].view(torch.int32)}
    if op == "attend":
        if own:
            _pool(s).attention(s["layer"], s["q"], s["out"], cu=s["cu"], max_new=s["max_new"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        out, lse = _attend(s)
        return {"out": out, "lse": lse}
    if op == "sparse":
        if own:
            p = _pool(s)
            p.select(s["layer"], s["q"], s["sel"], keep_first=1, keep_last=1)
            p.attention(s["layer"], s["q"], s["out"], sel=s["sel"])
            return {"out": s["out"], "sel": s["sel"]}
        sel = _choose(s)
        return {"out": _attend(s, sel)[0], "sel": sel}
    a, b = s["sides"][s["at"]], s["sides"][1 - s["at"]]
    fork, resize, compact = (_pool(s).fork, _pool(s).resize, _pool(s).compact) if own else (
        lambda *x: _fork(s, *x), lambda *x: _resize(s, *x), lambda: _compact(s))
    if op == "fork":
        resize(a, s["back"])               # the last step's tokens go again, so that every pass is the same step
        fork(s["sources"][s["at"]], b)
        resize(a, s["none"])
        resize(b, s["longer"])
    else:
        resize(a, s["none"])
        compact()
        resize(a, s["back"])
    s["at"] = 1 - s["at"]
    return {"pages": s["pages"].view(torch.int32), "summary": s["summary"].view(torch.int32), "table": s["table"],
            "seq_len": s["seq_len"], "refs": s["refs"]}


# ---- exact values, in 64 bits ----------------------------------------------------------------------------------------
def _e4m3(byte):
    e, m = (byte >> 3) & 15, byte & 7
    return torch.where(e == 0, m.double() * 2.0 ** -9, (1 + m.double() / 8) * torch.exp2(e.double() - 7))


def _e2m1(code):
    m, one = code & 7, code & 1
    size = torch.where(m < 2, m.double() / 2, (1 + one.double() / 2) * torch.exp2((m >> 1).double() - 1))
    return torch.where(code >= 8, -size, size)


def _token_values(s, row, pos):
    """Keys and values [n, hkv, d] of tokens `pos` of `row`, byte by byte."""
    c = s["case"]
    P, d, hkv = c["page"], c["d"], c["hkv"]
    b = min(P, 64)
    raw = s["pages"][s["layer"]].view(-1)
    page = s["table"][row, pos // P].long()
    t = (pos % P % b).view(-1, 1, 1)
    base = (((page.view(-1, 1, 1) * hkv + torch.arange(hkv, device=raw.device).view(1, -1, 1)) * (P // b)
             + (pos % P // b).view(-1, 1, 1)) * (b * d * 9 // 8))
    ch = torch.arange(d, device=raw.device).view(1, 1, -1)
    kb, ks = raw[base + t * (d // 2) + ch // 2].int(), raw[base + b * d // 2 + t * (d // 16) + ch // 16].int()
    k = _e2m1((kb >> (4 * (ch % 2))) & 15) * _e4m3(ks) * 2.0 ** c["k_exp"]
    base = base + b * d * 9 // 16
    group = ((t // 8) * (d // 16) + ch // 16) * 4 + t % 8 // 2
    vb, vs = raw[base + group * 16 + ch % 16].int(), raw[base + b * d // 2 + group * 2 + t % 2].int()
    return k, _e2m1((vb >> (4 * (t % 2))) & 15) * _e4m3(vs) * 2.0 ** c["v_exp"]


def _nearest(x, exp):
    """x in 64 bits as 16 channels' e4m3 scale and e2m1 codes hold it."""
    b = x.unflatten(-1, (-1, 16)) * 2.0 ** -exp
    t = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    t = torch.round(t / step) * step
    y = torch.where(t > 0, b / torch.where(t > 0, t, 1.0), 0.0).clamp(-6, 6)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)
    return (torch.round(y / step) * step * t).flatten(-2) * 2.0 ** exp


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # copies and whole numbers alone
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        return {"k": _nearest(s["k"].double(), c["k_exp"]), "v": _nearest(s["v"].double(), c["v_exp"]), "pages": None, "summary": None}
    g, d, P = c["g"], c["d"], c["page"]
    sel = _choose(s).long() if c["op"] == "sparse" else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for r, (n, m) in enumerate(zip(s["lens"], s["new"])):
        if n:
            pos = torch.arange(n, device="cuda")
            k, v = _token_values(s, torch.full_like(pos, r), pos)
            seen = pos <= torch.arange(n - m, n, device="cuda").view(-1, 1)
            for h in range(c["hkv"] * g):
                z = s["q"][at:at + m, h].double() @ k[:, h // g].T / math.sqrt(d)
                ok = seen if sel is None else seen & (pos // P == sel[r, h // g].view(-1, 1)).any(0)
                z = z.masked_fill(~ok, -math.inf)
                lse[at:at + m, h] = torch.logsumexp(z, -1)
                out[at:at + m, h] = torch.softmax(z, -1) @ v[:, h // g]
        at += m
    return {"out": out, "lse": lse} if sel is None else {"out": out, "sel": None}
