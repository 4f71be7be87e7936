"""More of the paged 4-bit cache's operators as a serving program calls them: cases, inputs, plain forms and exact values.

  cross   attention of a decoder's tokens over all of an encoder's states, which a row of the pool holds
  shared  attention of groups of rows that begin with the same pages: what they share is read and computed once for all
  weigh   add the attention weight that each held token gets from the newest queries to its score
  evict   of each row the tokens with the highest scores, for each layer and KV head, into the pages of a new row

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


# ---- cases -----------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(op=op, dtype="bf16", d=128, hkv=8, g=4, page=64, layers=1, rows=1, lo=1, hi=1, new_lo=1, new_hi=1, empty=0,
             members=1, pre_lo=0, pre_hi=0, keep=1, first=4, last=32, k_exp=0, v_exp=-2, salt=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one transcription's next token over its encoder's 1500 states, heads of 64 without groups: latency alone
        _case("cross 1x1 s1500 d64", "cross", dtype="f16", d=64, g=1, lo=1500, hi=1500, v_exp=0, salt=1),
        # 32 requests of up to 5 beams over states of ragged lengths, two rows of the batch are padding
        _case("cross 32x5 ragged d64", "cross", dtype="f16", d=64, hkv=16, g=1, page=32, rows=32, lo=37, hi=1500, new_lo=3,
              new_hi=5, empty=2, v_exp=0, salt=2),
        # decoder prompts over long documents, the largest batch of products
        _case("cross 4x1024 s16384", "cross", rows=4, lo=12001, hi=16384, new_lo=700, new_hi=1024, salt=3),
        # 8 samples of one prompt, four layers of a decode step
        _case("shared 1x8 s2000", "shared", layers=4, rows=1, members=8, pre_lo=2000, pre_hi=2000, lo=1, hi=90, salt=4),
        # a full batch behind one long instruction, four layers of a decode step
        _case("shared 1x64 s8192", "shared", layers=4, rows=1, members=64, pre_lo=8192, pre_hi=8192, lo=16, hi=500, salt=5),
        # 8 documents with up to 16 readers each, small pages, 8 query heads for each KV head
        _case("shared 8x16 ragged f16 p16 g8", "shared", dtype="f16", hkv=4, g=8, page=16, layers=2, rows=8, members=16,
              pre_lo=500, pre_hi=12000, lo=1, hi=700, empty=1, salt=6),
        # questions of up to 24 tokens over one document
        _case("shared 1x32 s16384 n24", "shared", rows=1, members=32, pre_lo=16384, pre_hi=16384, lo=24, hi=400, new_lo=9,
              new_hi=24, salt=7),
        # the decode step of a batch at its budget
        _case("weigh 16x1 s4160", "weigh", rows=16, lo=4160, hi=4160, salt=8),
        # the last 64 queries of long prompts say what to keep of them
        _case("weigh 4x64 s16384", "weigh", dtype="f16", page=32, rows=4, lo=9001, hi=16384, new_lo=64, new_hi=64, salt=9),
        # every query of a prompt's chunk has its say
        _case("weigh 1x2048 s16384", "weigh", lo=16384, hi=16384, new_lo=2048, new_hi=2048, salt=10),
        # a batch goes back to its budget, two layers
        _case("evict 16 rows 4160 to 4096", "evict", layers=2, rows=16, lo=4160, hi=4160, keep=4096, salt=11),
        # prompts of ragged lengths keep an eighth, eight layers
        _case("evict 4 prompts to 2048", "evict", layers=8, rows=4, lo=9001, hi=16384, keep=2048, last=64, salt=12),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["cross", "shared", "weigh", "evict"])
        kw = dict(dtype=rng.choice(["bf16", "f16"]), d=rng.choice([64, 128, 128]), hkv=rng.choice([1, 2, 4, 8, 16]),
                  g=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]), page=rng.choice([16, 32, 64, 128]), salt=rng.randrange(1 << 20),
                  k_exp=rng.choice([0, 0, 2, -3]), v_exp=rng.choice([0, -2, -5]), layers=rng.choice([1, 1, 2, 3]))
        if op == "cross":
            kw.update(rows=size(1, 64), hi=size(1, 16384), new_hi=rng.choice([1, size(2, 16), size(17, 1024)]), empty=rng.choice([0, 0, 2]))
        elif op == "shared":
            kw.update(rows=size(1, 16), members=size(1, 64), pre_hi=size(16, 16384), hi=size(1, 1000), empty=rng.choice([0, 0, 1]),
                      new_hi=rng.choice([1, 1, size(2, 32)]))
            kw["pre_lo"] = max(1, int(kw["pre_hi"] * rng.choice([0.1, 1.0])))
        elif op == "weigh":
            kw.update(rows=size(1, 64), hi=size(1, 16384), new_hi=rng.choice([1, 1, size(2, 64), size(65, 2048)]), empty=rng.choice([0, 0, 1]))
        else:
            kw.update(rows=size(1, 32), hi=size(64, 16384), first=rng.choice([0, 4]), last=rng.choice([0, 16, 64]))
            kw["keep"] = max(68, int(kw["hi"] * rng.choice([0.1, 0.5, 0.98])))
        kw["lo"] = max(1, int(kw["hi"] * rng.choice([0.05, 0.5, 1.0])))
        kw["new_lo"] = max(1, int(kw.get("new_hi", 1) * rng.choice([0.1, 1.0])))
        c = _case("", op, **kw)
        if _cost(c) <= most and _held(c) <= 40e9:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280)  # this card's flops for each byte


def _held(c):
    """Bytes that the plain form keeps at once, about."""
    sh = _shape(c)
    heads, hq = c["layers"] * c["hkv"] * c["d"], c["layers"] * c["hkv"] * c["g"]
    n, most = len(sh["lens"]), max(sh["lens"])
    if c["op"] == "shared":
        per = max(sum(sh["new"][a:b]) for a, b in sh["groups"])
        tail = max(x - y for x, y in zip(sh["lens"], sh["prefix"])) + c["page"]
        return (c["rows"] * max(sh["prefix"]) + n * tail) * heads * 40 + hq * 12 * (c["rows"] * per * max(sh["prefix"]) + n * max(sh["new"]) * tail)
    return n * most * heads * 40 + n * max(sh["new"]) * hq * most * 12


def _shape(c):
    """Lengths (with the new tokens), new tokens or queries, groups of rows and what each row shares with its group."""
    rng = random.Random(c["salt"] * 7 + 1)
    if c["op"] != "shared":
        n = c["rows"]
        lens = [rng.randint(c["lo"], c["hi"]) for _ in range(n)]
        if n > 2:
            lens[0], lens[n // 2] = c["hi"], c["lo"]
        new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(n)]
        if c["op"] == "weigh":
            new = [min(a, b) for a, b in zip(lens, new)]
        if c["empty"] and n > c["empty"]:  # rows of a padded batch: queries, and nothing in the cache
            lens[-c["empty"]:] = [0] * c["empty"]
            new[-c["empty"]:] = [1] * c["empty"]
        return dict(lens=lens, new=new, groups=[(i, i + 1) for i in range(n)], prefix=[0] * n)
    lens, new, groups, prefix = [], [], [], []
    for _ in range(c["rows"]):
        m = c["members"] if c["rows"] == 1 else rng.randint(max(1, c["members"] // 3), c["members"])
        p = rng.randint(c["pre_lo"], c["pre_hi"])
        groups.append((len(lens), len(lens) + m))
        for i in range(m):
            y = rng.randint(c["new_lo"], c["new_hi"])
            lens.append(p + max(y, rng.randint(c["lo"], c["hi"])))
            new.append(y)
            prefix.append(p // c["page"] * c["page"])
        if c["empty"] and m > 2:  # a place of the group that nobody has
            lens[-1], new[-1] = 0, 1
    return dict(lens=lens, new=new, groups=groups, prefix=prefix)


def _page_bytes(c):
    return c["page"] * c["d"] * 9 // 8


def _pages(c, n):
    return -(-n // c["page"])


def _kept(c, lens):
    return [min(x, c["keep"]) for x in lens]


def work(c):
    sh = _shape(c)
    lens, new = sh["lens"], sh["new"]
    d, hkv, hq, L = c["d"], c["hkv"], c["hkv"] * c["g"], c["layers"]
    tok, n = hkv * d * 9 // 8, sum(new)  # bytes of a token's keys and values
    if c["op"] == "cross":
        return {"bytes": 4 * n * hq * d + 4 * n * hq + sum(lens) * tok + 4 * sum(_pages(c, x) for x in lens),
                "flops": 4 * sum(x * y for x, y in zip(lens, new)) * hq * d}
    pairs = sum(y * x - y * (y - 1) // 2 for x, y in zip(lens, new) if x)
    if c["op"] == "shared":
        held = sum(sh["prefix"][a] for a, _ in sh["groups"]) + sum(x - y for x, y in zip(lens, sh["prefix"]) if x)
        return {"bytes": L * (4 * n * hq * d + 4 * n * hq + held * tok) + 4 * sum(_pages(c, x) for x in lens),
                "flops": 4 * L * pairs * hq * d}
    if c["op"] == "weigh":
        held = sum(lens)
        return {"bytes": 2 * n * hq * d + 4 * n * hq + held * tok // 2 + 4 * hkv * (2 * held - n) + 4 * sum(_pages(c, x) for x in lens),
                "flops": 2 * pairs * hq * d}
    keep = _kept(c, lens)
    return {"bytes": L * (hkv * 4 * (sum(lens) + sum(keep)) + 2 * sum(keep) * tok + sum(_pages(c, x) for x in keep) * hkv * (2 * d + 4)),
            "flops": 0}


# ---- the page format, in torch -----------------------------------------------------------------------------------
def _quantise(x, exp):
    """x [..., d] in 32 bits -> codes [..., d], scales [..., d / 16] (e4m3)."""
    b = x.unflatten(-1, (-1, 16))
    top = b.abs().amax(-1)
    s = (top / 6.0 * 2.0 ** -exp).clamp(max=448.0).to(torch.float8_e4m3fn)
    S = s.float().unsqueeze(-1) * 2.0 ** exp
    a = b.abs()
    code = ((a > 0.25 * S).byte() + (a >= 0.75 * S).byte() + (a > 1.25 * S).byte() + (a >= 1.75 * S).byte()
            + (a > 2.5 * S).byte() + (a >= 3.5 * S).byte() + (a > 5.0 * S).byte())
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


def _values(code, scale, exp):
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    x = torch.cat([m, -m])[code.int()].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)
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
    sh = _shape(c)
    lens, new, groups, prefix = sh["lens"], sh["new"], sh["groups"], sh["prefix"]
    R, P, d, hkv, L = len(lens), c["page"], c["d"], c["hkv"], c["layers"]
    hq, n = hkv * c["g"], sum(new)
    keep = _kept(c, lens)
    i32 = dict(dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # which pages: what a group shares, then each row's own
    entries, at = [], 0
    for a, b in groups:
        common = prefix[a] // P
        for i in range(a, b):
            entries += [(i, j, at + j) for j in range(min(common, _pages(c, lens[i])))]
        at += common
    for i in range(R):
        for j in range(prefix[i] // P, _pages(c, lens[i])):
            entries.append((i, j, at))
            at += 1
    M = max(1, max(_pages(c, x) for x in lens))
    N = at + 3 + (sum(_pages(c, x) for x in keep) if c["op"] == "evict" else 0)
    order = torch.randperm(N, generator=gen, device=dev).int()
    where = torch.tensor(entries, dtype=torch.int64, device=dev)
    table = torch.full((2 * R if c["op"] == "evict" else R, M), -1, **i32)
    table[where[:, 0], where[:, 1]] = order[where[:, 2]]
    refs = torch.bincount(order[where[:, 2]].long(), minlength=N).int()

    # keys with a mean of their own in every channel and a few channels ten times as large, as projections give them
    mean, wide = normal(hkv, 1, d) * math.sqrt(2.0), torch.ones(hkv, 1, d, device=dev)
    wide.view(-1)[torch.randperm(hkv * d, generator=gen, device=dev)[: max(1, hkv * d // 100)]] = 10.0
    pages = torch.empty(L, N, hkv, _page_bytes(c), dtype=torch.uint8, device=dev)
    summary = torch.empty(L, N, hkv, 2 * d + 16, dtype=torch.uint8, device=dev)
    for layer in range(L):
        for part in range(0, N, 512):  # a part of the pool at a time
            m = min(512, N - part)
            kc, ks = _quantise((normal(m, hkv, P, d) + mean) * wide, c["k_exp"])
            vc, vs = _quantise(normal(m, hkv, P, d) * 2.0 ** (c["v_exp"] + 2), c["v_exp"])
            pages[layer, part:part + m] = _pack(kc, ks, vc, vs)
            summary[layer, part:part + m] = _summary(_values(kc, ks, 0), torch.full((m, hkv), P, device=dev))
    size = torch.tensor(lens + [0] * (table.shape[0] - R), **i32)
    s = {"case": c, "lens": lens, "new": new, "groups": groups, "max_new": max(new), "pages": pages, "summary": summary,
         "table": table, "seq_len": size, "refs": refs, "prefix": prefix}
    s["cu"] = None if max(new) == min(new) == 1 else torch.tensor([sum(new[:i]) for i in range(R + 1)], **i32)
    s["row"] = torch.tensor([i for i, y in enumerate(new) for _ in range(y)], device=dev)
    s["turn"] = torch.tensor([t for y in new for t in range(y)], device=dev)
    # the last token that each query sees
    seen = [x - 1 if c["op"] == "cross" else x - y + t for x, y in zip(lens, new) for t in range(y)]
    s["pos"] = torch.tensor(seen, device=dev)
    if c["op"] != "evict":
        s["q"] = normal(L, n, hq, d).to(DTYPES[c["dtype"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(L, n, hq, dtype=torch.float32, device=dev)
    if c["op"] == "shared":
        s["bounds"] = torch.tensor([a for a, _ in groups] + [R], **i32)
        s["max_group"] = max(sum(new[a:b]) for a, b in groups)
        s["plan"] = torch.empty(R, 2, **i32)
        s["of"] = torch.tensor([k for k, (a, b) in enumerate(groups) for _ in range(a, b)], device=dev)  # a row's group
        s["in_group"] = torch.tensor([i - sum(new[:a]) for a, b in groups for i in range(sum(new[:a]), sum(new[:b]))], device=dev)
    if c["op"] == "weigh":
        score, top = _logits(s, s["table"].unsqueeze(0))
        score = torch.where(top == -math.inf, -math.inf, (score - torch.where(top == -math.inf, 0.0, top)).exp().sum(-1, keepdim=True).log() + top)
        s["lse"].copy_(_of_tokens(s, score)[..., 0])
        s["scores"] = torch.rand(L, R, hkv, M * P, generator=gen, device=dev)
    if c["op"] == "evict":
        # most tokens are worth next to nothing, some are not there yet (0): accumulated weights as a few hundred queries give them
        s["scores"] = torch.exp(2.0 * normal(L, 2 * R, hkv, M * P) - 3.0)
        s["scores"] *= torch.rand(s["scores"].shape, generator=gen, device=dev) > 0.1
        s["src"], s["dst"] = torch.arange(R, **i32), torch.arange(R, 2 * R, **i32)
        s["keep"], s["none"] = torch.tensor(keep, **i32), torch.zeros(R, **i32)
        s["kept"] = keep
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
        if c["op"] == "shared":
            s["scratch"] = s["pool"].shared_scratch(s["q"].shape[1])
    return s["pool"]


def _own(s):
    p, op, c = _pool(s), s["case"]["op"], s["case"]
    kw = dict(cu=s["cu"], max_new=s["max_new"])
    if op == "evict":
        p.resize(s["dst"], s["none"])  # the last pass's rows go
        p.resize(s["dst"], s["keep"])
        p.evict(s["scores"], s["src"], s["dst"], keep_first=c["first"], keep_last=c["last"])
        return
    if op == "shared":
        p.common(s["plan"], groups=s["bounds"], cu=s["cu"])
    for layer in range(c["layers"]):
        q, out, lse = s["q"][layer], s["out"][layer], s["lse"][layer]
        if op == "cross":
            p.cross(layer, q, out, lse=lse, **kw)
        elif op == "shared":
            p.shared(layer, q, out, s["plan"], s["scratch"], groups=s["bounds"], max_group=s["max_group"], lse=lse, **kw)
        else:
            p.weigh(layer, q, lse, s["scores"][layer], **kw)


# ---- the plain forms ---------------------------------------------------------------------------------------------------
def _tokens(s, table):
    """Keys and values [L, rows, hkv, S, d] in 32 bits of the pages that table [1, rows, M] names (any page where it is -1)."""
    c = s["case"]
    raw = s["pages"][:, table[0].clamp(min=0).long()]  # [L, rows, M, hkv, bytes]
    kc, ks, vc, vs = _codes(raw.transpose(2, 3), c["page"], c["d"])
    return _values(kc, ks, c["k_exp"]).flatten(3, 4), _values(vc, vs, c["v_exp"]).flatten(3, 4)


def _of_tokens(s, x):
    """x [L, rows, hkv, T g, any] -> [L, n, hq, any]: the queries that there are."""
    c = s["case"]
    x = x.unflatten(3, (s["max_new"], c["g"])).transpose(2, 3)
    return x[:, s["row"], s["turn"]].flatten(2, 3)


def _by_rows(s, row, turn, rows, most):
    """The queries in 32 bits as [L, rows, hkv, most g, d]."""
    c = s["case"]
    q = torch.zeros(c["layers"], rows, most, c["hkv"], c["g"], c["d"], device=row.device)
    q[:, row, turn] = s["q"].float().unflatten(2, (c["hkv"], c["g"]))
    return q.permute(0, 1, 3, 2, 4, 5).flatten(3, 4)


def _logits(s, table, k=None):
    """Logits [L, R, hkv, T g, S] of each row's queries (-inf where they do not look) and their largest."""
    c = s["case"]
    k = _tokens(s, table)[0] if k is None else k
    R, S, T = table.shape[1], k.shape[3], s["max_new"]
    score = torch.matmul(_by_rows(s, s["row"], s["turn"], R, T), k.transpose(-1, -2)).mul_(c["d"] ** -0.5)
    last = torch.full((R, T), -1, device=k.device)
    last[s["row"], s["turn"]] = s["pos"]
    hidden = torch.arange(S, device=k.device) > last.unsqueeze(-1)  # [R, T, S]
    score.masked_fill_(hidden.repeat_interleave(c["g"], 1).view(1, R, 1, T * c["g"], S), -math.inf)
    return score, score.amax(-1, keepdim=True)


def _cross(s):
    k, v = _tokens(s, s["table"].unsqueeze(0))
    score, top = _logits(s, s["table"].unsqueeze(0), k)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(_of_tokens(s, out))
    s["lse"].copy_(_of_tokens(s, top + total.log())[..., 0])


def _shared(s):
    """Logits over what the group's tables have in common, one product for the group, beside those over the row's own
    pages; one softmax over both."""
    c = s["case"]
    P, g, dev = c["page"], c["g"], s["table"].device
    table, of = s["table"], s["of"]
    R, M, G = table.shape[0], table.shape[1], len(s["groups"])
    there = s["seq_len"] > 0
    new = torch.bincount(s["row"], minlength=R)
    # whole leading pages that all of a group's rows have (its places that nobody has do not count)
    leader = torch.full((G,), R - 1, device=dev).scatter_reduce(0, of, torch.where(there, torch.arange(R, device=dev), R - 1), "amin")
    same = ((table == table[leader[of]]) & (torch.arange(M, device=dev) < ((s["seq_len"] - new) // P).unsqueeze(1))).int()
    run_ = torch.where(there, same.cumprod(1).sum(1), M)
    common = torch.full((G,), M, device=dev).scatter_reduce(0, of, run_, "amin")
    m = max(1, max(s["prefix"]) // P)
    common = torch.where(common < M, common, 0).clamp(max=m)  # (a row alone shares all with itself)
    # over the common pages
    k, v = _tokens(s, table[leader, :m].unsqueeze(0))
    most = s["max_group"]
    q = _by_rows(s, of[s["row"]], s["in_group"], G, most)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(c["d"] ** -0.5)
    z.masked_fill_((torch.arange(m * P, device=dev) >= (common * P).unsqueeze(1)).view(1, G, 1, 1, m * P), -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    parts = torch.cat([torch.matmul(p, v), p.sum(-1, keepdim=True), top], -1)
    parts = parts.unflatten(3, (most, g)).transpose(2, 3)[:, of[s["row"]], s["in_group"]].flatten(2, 3)  # [L, n, hq, d + 2]
    # over the rows' own pages
    width = max(1, max(_pages(c, x) - y // P for x, y in zip(s["lens"], s["prefix"])))
    j = torch.arange(width, device=dev) + common[of].unsqueeze(1)
    mine = torch.where(j < M, table.gather(1, j.clamp(max=M - 1)), -1)
    k, v = _tokens(s, mine.unsqueeze(0))
    T, S = s["max_new"], width * P
    z = torch.matmul(_by_rows(s, s["row"], s["turn"], R, T), k.transpose(-1, -2)).mul_(c["d"] ** -0.5)
    last = torch.full((R, T), -1, device=dev)
    last[s["row"], s["turn"]] = s["pos"]
    at = torch.arange(S, device=dev) + (common[of] * P).unsqueeze(1)
    hidden = at.unsqueeze(1) > last.unsqueeze(-1)
    z.masked_fill_(hidden.repeat_interleave(g, 1).view(1, R, 1, T * g, S), -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    mine = _of_tokens(s, torch.cat([torch.matmul(p, v), p.sum(-1, keepdim=True), top], -1))
    # both together
    nobody = (s["seq_len"] == 0)[s["row"]].view(1, -1, 1, 1)
    a, la, ma = parts.split([c["d"], 1, 1], -1)
    b, lb, mb = mine.split([c["d"], 1, 1], -1)
    ma = torch.where(nobody, -math.inf, ma)
    top = torch.maximum(ma, mb)
    base = torch.where(top == -math.inf, 0.0, top)
    wa, wb = (ma - base).exp(), (mb - base).exp()
    total = la * wa + lb * wb
    s["out"].copy_((a * wa + b * wb) / torch.where(total == 0, 1.0, total))
    s["lse"].copy_((top + total.log())[..., 0])


def _weigh(s):
    c = s["case"]
    score, _ = _logits(s, s["table"].unsqueeze(0))
    R, T = s["table"].shape[0], s["max_new"]
    lse = torch.full((c["layers"], R, T, c["hkv"], c["g"]), math.inf, device=score.device)
    lse[:, s["row"], s["turn"]] = torch.where(s["lse"] == -math.inf, math.inf, s["lse"]).unflatten(2, (c["hkv"], c["g"]))
    got = score.sub_(lse.permute(0, 1, 3, 2, 4).flatten(3).unsqueeze(-1)).exp_().sum(3)  # [L, R, hkv, S]
    new = torch.bincount(s["row"], minlength=R)
    j = torch.arange(got.shape[-1], device=got.device)
    held = s["seq_len"].view(1, R, 1, 1)
    old = torch.where(j < held - new.view(1, R, 1, 1), s["scores"], 0.0)
    s["scores"].copy_(torch.where(j < held, old + got, s["scores"]))


def _take_pages(s):
    """Rows dst give their pages back, then each in turn takes the lowest free pages for what it is to hold."""
    P, dst = s["case"]["page"], s["dst"].long()
    t = s["table"][dst]
    s["refs"] -= torch.bincount(t[t >= 0].long(), minlength=s["refs"].shape[0]).int()
    free = (s["refs"] == 0).nonzero().squeeze(1).int()
    has = (s["keep"] + P - 1) // P
    first = (has.cumsum(0) - has).unsqueeze(1)
    j = torch.arange(t.shape[1], device=t.device)
    t = torch.where(j < has.unsqueeze(1), free[(first + j).clamp(max=len(free) - 1)], -1)
    s["refs"][t[t >= 0].long()] = 1
    s["table"][dst], s["seq_len"][dst] = t, s["keep"]


def _evict(s):
    c = s["case"]
    P, d, dev = c["page"], c["d"], s["table"].device
    _take_pages(s)
    src, dst = s["src"].long(), s["dst"].long()
    S, width = s["table"].shape[1] * P, max(1, max(_pages(c, x) for x in s["kept"]))
    # the kept tokens, ascending, for each layer, row and KV head
    size = s["seq_len"][src].view(1, -1, 1, 1)
    j = torch.arange(S, device=dev)
    score = s["scores"][:, src]
    worth = torch.where((j < c["first"]) | (j >= size - c["last"]), math.inf, score)
    worth = torch.where(j < size, worth, -math.inf)
    best = torch.sort(worth, dim=-1, descending=True, stable=True).indices[..., : width * P]
    k = torch.arange(best.shape[-1], device=dev)
    count = s["keep"].view(1, -1, 1, 1)
    best = torch.where(k < count, best, S).sort(-1).values.clamp(max=S - 1)
    best = torch.nn.functional.pad(best, (0, width * P - best.shape[-1]))  # (a page past the source's)
    # their codes and scales, page by page
    codes = _codes(s["pages"][:, s["table"][src].clamp(min=0).long()].transpose(2, 3), P, d)
    to = s["table"][dst, :width]
    ids = to.clamp(min=0).long()
    old = _codes(s["pages"][:, ids].transpose(2, 3), P, d)  # [L, R, hkv, width, P, .]
    inside = (torch.arange(width * P, device=dev) < count).unsqueeze(-1)
    now = []
    for x, y in zip(codes, old):
        got = x.view(torch.uint8).flatten(3, 4).gather(3, best.unsqueeze(-1).expand(*best.shape, x.shape[-1]))
        now.append(torch.where(inside, got, y.view(torch.uint8).flatten(3, 4)).unflatten(3, (width, P)))
    taken = to >= 0
    s["pages"][:, to[taken].long()] = _pack(*now).transpose(2, 3)[:, taken]
    held = (s["keep"].unsqueeze(1) - torch.arange(width, device=dev) * P).clamp(1, P)
    sums = _summary(_values(now[0], now[1].view(torch.float8_e4m3fn), 0), held.view(1, -1, 1, width).expand(now[0].shape[:4]))
    s["summary"][:, to[taken].long()] = sums.transpose(2, 3)[:, taken]
    m = min(S, width * P)
    s["scores"][:, dst, :, :m] = torch.where(inside[..., :m, 0], score.gather(3, best[..., :m]), s["scores"][:, dst, :, :m])


def run(s):
    op = s["case"]["op"]
    if own:
        _own(s)
    else:
        {"cross": _cross, "shared": _shared, "weigh": _weigh, "evict": _evict}[op](s)
    if op in ("cross", "shared"):
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weigh":
        return {"scores": s["scores"]}
    return {"pages": s["pages"].view(torch.int32), "summary": s["summary"].view(torch.int32), "table": s["table"],
            "seq_len": s["seq_len"], "refs": s["refs"], "scores": s["scores"].view(torch.int32)}


# ---- exact values, in 64 bits ----------------------------------------------------------------------------------------
def _e4m3(byte):
    e, m = (byte >> 3) & 15, byte & 7
    return torch.where(e == 0, m.double() * 2.0 ** -9, (1 + m.double() / 8) * torch.exp2(e.double() - 7))


def _e2m1(code):
    m, one = code & 7, code & 1
    size = torch.where(m < 2, m.double() / 2, (1 + one.double() / 2) * torch.exp2((m >> 1).double() - 1))
    return torch.where(code >= 8, -size, size)


def _held_row(s, layer, row, n):
    """Keys and values [n, hkv, d] of a row's tokens, byte by byte."""
    c = s["case"]
    P, d, hkv = c["page"], c["d"], c["hkv"]
    b = min(P, 64)
    raw = s["pages"][layer].view(-1)
    pos = torch.arange(n, device=raw.device)
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


def exact(case, seed):
    if case["op"] == "evict":
        return None  # a choice and copies alone
    s = prepare(case, seed)
    c = s["case"]
    g, d = c["g"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if c["op"] == "weigh" else None
    for layer in range(c["layers"]):
        at = 0
        for r, (n, m) in enumerate(zip(s["lens"], s["new"])):
            if n:
                k, v = _held_row(s, layer, r, n)
                hidden = torch.arange(n, device="cuda") > s["pos"][at:at + m].view(-1, 1)
                for h in range(c["hkv"] * g):
                    z = s["q"][layer, at:at + m, h].double() @ k[:, h // g].T / math.sqrt(d)
                    z = z.masked_fill(hidden, -math.inf)
                    if scores is not None:
                        if h % g == 0:
                            scores[layer, r, h // g, n - m:n] = 0
                        scores[layer, r, h // g, :n] += torch.exp(z - s["lse"][layer, at:at + m, h].double().view(-1, 1)).sum(0)
                        continue
                    lse[layer, at:at + m, h] = torch.logsumexp(z, -1)
                    out[layer, at:at + m, h] = torch.softmax(z, -1) @ v[:, h // g]
            at += m
    return {"scores": scores} if scores is not None else {"out": out, "lse": lse}
