"""Cases of the 4-bit KV cache, of decode attention that records its weights, and of eviction.

Four operators:
  * "append":  this step's (or a prompt chunk's) K and V rows into a cache held in 4 bits, read back as
               the fp16 values that the codes stand for;
  * "int4":    decode attention over such a cache, one query token per sequence or a few;
  * "weights": decode attention that also adds every key's softmax weight to a running total per key;
  * "evict":   the cache cut to a budget of tokens per KV head by that total, kept rows moved in order.

``run`` computes them in elementary torch operations, or, with ``own``, by the package's entry points.
"""
import math

import torch

own = False

BLOCK = 32          # head_dim elements per scale of the 4-bit cache


# --------------------------------------------------------------------------- cases
def listed():
    def case(name, op, batch, hq, hkv, d, lo, hi, **more):
        c = {"name": name, "op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "lo": lo, "hi": hi,
             "tq": 1, "paged": True, "window": 0, "int4": op in ("append", "int4"), "budget": 0}
        c.update(more)
        return c

    return [
        # one decode step's rows of 64 sequences: a call that is all latency
        case("append_64x1_d128", "append", 64, 32, 8, 128, 1, 1),
        # a prompt's chunk of 8 sequences written into the cache and read back for the next chunk
        case("append_8x2048_d128", "append", 8, 32, 8, 128, 2048, 2048),
        # the smallest decode step: one short chat
        case("int4_1x512_d128", "int4", 1, 8, 2, 128, 512, 512, paged=False),
        # a few sequences of mixed length, head_dim 256
        case("int4_4x1k-8k_d256", "int4", 4, 16, 8, 256, 1024, 8192, paged=False),
        # long-context serving: the workload that 4 bits are for
        case("int4_32x32k_d128", "int4", 32, 32, 8, 128, 32768, 32768),
        # drafts of 4 tokens verified at once, odd ragged lengths, sliding windows on odd sequences
        case("int4_16x5k-16k_d128_4q", "int4", 16, 32, 4, 128, 5003, 16381, tq=4, window=4096),
        # one short sequence whose weights are recorded
        case("weights_1x512_d128", "weights", 1, 8, 2, 128, 512, 512, paged=False),
        # every step of a served batch recorded, fp16 cache
        case("weights_16x16k_d128", "weights", 16, 32, 8, 128, 16384, 16384),
        # a prompt's last 32 tokens as the observers, over a cache held in 4 bits, ragged
        case("weights_8x1k-9k_d256_32q_int4", "weights", 8, 16, 8, 256, 1021, 9001, tq=32, int4=True),
        # one short sequence cut in half
        case("evict_1x1000_d128", "evict", 1, 8, 2, 128, 1000, 1000, paged=False, budget=512),
        # a served batch cut to 2048 tokens, ragged, some sequences already short enough
        case("evict_32x1k-8k_d128", "evict", 32, 32, 8, 128, 1024, 8192, budget=2048),
        # one long document cut to an eighth
        case("evict_1x128k_d256", "evict", 1, 16, 8, 256, 131072, 131072, budget=16384),
    ]


def draw(rng):
    def spread(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["append", "int4", "weights", "evict"])
    d = rng.choice([128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    c = {"op": op, "d": d, "hkv": hkv, "hq": hq, "tq": 1, "window": 0, "budget": 0,
         "paged": rng.random() < 0.7, "int4": op in ("append", "int4")}
    if op == "append":
        c["batch"] = spread(1, 64)
        c["lo"] = c["hi"] = spread(1, max(1, 1 << 14) // c["batch"] + 1)
        return c
    c["batch"] = spread(1, 48)
    hi = spread(100, min(65536, (1 << 20) // (c["batch"] * (d // 128))))
    if op == "weights":
        hi = max(100, hi // 4)
        c["int4"] = rng.random() < 0.5
    c["hi"] = hi
    c["lo"] = max(1, int(hi * rng.choice([1.0, 0.5, 0.05])))
    if op != "evict":
        c["tq"] = rng.choice([1, 1, 1, 2, 3, 5])
        c["window"] = rng.choice([0, 0, spread(16, hi)])
    else:
        c["budget"] = max(8, int(hi * rng.uniform(0.1, 0.9)))
    return c


def lens_of(case):
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def pins_of(case):
    """(first, last) tokens of a sequence that eviction always keeps."""
    return min(4, case["budget"] // 4), case["budget"] // 4


def seen_of(case):
    """Keys each sequence's step reads."""
    got = []
    for b, n in enumerate(lens_of(case)):
        w = case["window"] if b % 2 else 0
        got.append(min(n, w + case["tq"] - 1) if w else n)
    return got


def work(case):
    b, hq, hkv, d, tq = case["batch"], case["hq"], case["hkv"], case["d"], case["tq"]
    if case["op"] == "append":
        rows = b * case["hi"] * hkv * 2
        return {"bytes": rows * (4 * d + 2 * (d // 2 + d // 16) + 2 * d), "flops": rows * d * 4}
    if case["op"] == "evict":
        moved = 0
        for n in lens_of(case):
            if n > case["budget"]:
                moved += (case["budget"] - pins_of(case)[0]) * hkv
        return {"bytes": moved * 2 * (4 * d + 4) + sum(lens_of(case)) * hkv * 4, "flops": 0}
    keys = sum(seen_of(case)) * hkv
    row = 2 * (d // 2 + d // 16) if case["int4"] else 4 * d
    more = 8 if case["op"] == "weights" else 0
    return {"bytes": keys * (row + more) + b * tq * hq * d * 4, "flops": keys * 4 * d * (hq // hkv) * tq}


# --------------------------------------------------------------------------- the 4-bit rows
def pack(x):
    """fp32 [..., D] -> (codes uint8 [..., D/2], scales fp16 [..., D/32])."""
    d = x.shape[-1]
    blk = x.float().unflatten(-1, (d // BLOCK, BLOCK))
    s = (blk.abs().amax(-1) / 7.0).half()
    sf = s.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round(blk / sf), torch.zeros_like(blk)).clamp_(-7, 7)
    u = (c + 8).to(torch.uint8).unflatten(-1, (4, 4, 2))           # [..., j, octet, byte, nibble]
    by = u[..., 0] | (u[..., 1] << 4)                              # [..., j, octet, 4 bytes]
    return by.transpose(-3, -2).reshape(*x.shape[:-1], d // 2).contiguous(), s.contiguous()


def unpack(codes, scales):
    """The fp32 values that 4-bit rows stand for."""
    d = codes.shape[-1] * 2
    by = codes.reshape(*codes.shape[:-1], 4, d // BLOCK, 4).transpose(-3, -2)   # [..., j, octet, 4]
    c = torch.stack((by & 15, by >> 4), dim=-1).reshape(*codes.shape[:-1], d // BLOCK, BLOCK)
    return ((c.float() - 8.0) * scales.float().unsqueeze(-1)).reshape(*codes.shape[:-1], d)


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    b, hq, hkv, d, tq = case["batch"], case["hq"], case["hkv"], case["d"], case["tq"]
    lens = lens_of(case)
    page = 16
    at = 5 if case["op"] == "append" else 0                        # rows already in the cache
    blocks = -(-(max(lens) + at) // page)
    cap = blocks * page
    s = {"case": case, "page": page, "cap": cap, "scale": d ** -0.5,
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if case["paged"]:
        total = b * blocks + 3
        order = torch.randperm(total, generator=g, device=dev)[:b * blocks]
        s["table"] = order.to(torch.int32).view(b, blocks).contiguous()
        shape = (total, hkv, page)
    else:
        s["table"] = None
        shape = (b, hkv, cap)

    def rows():
        x = torch.empty(*shape, d, dtype=torch.float16, device=dev)
        return x.normal_(generator=g)

    if case["op"] == "append":
        for n in ("k", "v"):
            s[n + "_new"] = torch.randn(b, case["hi"], hkv, d, generator=g, device=dev).half().float()
            s[n] = torch.full((*shape, d // 2), 0x88, dtype=torch.uint8, device=dev)
            s[n + "s"] = torch.zeros(*shape, d // BLOCK, dtype=torch.float16, device=dev)
            s[n + "_out"] = torch.empty(b, case["hi"], hkv, d, dtype=torch.float16, device=dev)
        s["pos"] = torch.full((b,), at, dtype=torch.int32, device=dev)
        return s
    for n in ("k", "v"):
        if case["int4"]:
            s[n], s[n + "s"] = pack(rows())
        else:
            s[n], s[n + "s"] = rows(), None
    if case["op"] == "evict":
        # totals after a while of decoding: heavy-tailed, with the exact ties of tokens never looked at
        t = torch.rand(*shape, generator=g, device=dev)
        s["acc"] = torch.where(t < 0.1, torch.zeros_like(t), t.pow(8.0) * 50.0)
        s["new_lens"] = torch.empty_like(s["lens"])
        s["kept"] = torch.empty(b, hkv, case["budget"], dtype=torch.int32, device=dev)
        return s
    s["q"] = torch.randn(b, tq, hq, d, generator=g, device=dev).half()
    s["out"] = torch.empty(b, tq, hq, d, dtype=torch.float16, device=dev)
    w = case["window"]
    s["window"] = None
    if w:
        s["window"] = torch.tensor([w if i % 2 else 0 for i in range(b)], dtype=torch.int32, device=dev)
    if case["op"] == "weights":
        s["acc"] = torch.rand(*shape, generator=g, device=dev)
    if own:
        import decode_step_kv_gb300 as fa
        if case["int4"]:
            s["ws"] = fa.alloc_workspace_int4(b, tq, hq, hkv, d, cap, weights=case["op"] == "weights")
        else:
            s["ws"] = fa.alloc_workspace_weights(b, tq, hq, hkv, d, cap)
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": own_append, "int4": own_int4, "weights": own_weights, "evict": own_evict}[op](state)
    return {"append": plain_append, "int4": plain_attend, "weights": plain_attend, "evict": plain_evict}[op](state)


def own_append(s):
    import decode_step_kv_gb300 as fa
    fa.fa_append_kv_int4(s["k_new"], s["v_new"], s["k"], s["ks"], s["v"], s["vs"], s["table"], s["pos"])
    fa.fa_gather_kv_int4(s["k"], s["ks"], s["v"], s["vs"], s["table"], s["pos"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def own_int4(s):
    import decode_step_kv_gb300 as fa
    c = s["case"]
    fa.fa_decode_int4(s["q"], s["k"], s["ks"], s["v"], s["vs"], s["table"], s["lens"], c["hq"], c["hkv"], c["d"],
                      s["scale"], s["window"], s["out"], workspace=s["ws"])
    return s["out"]


def own_weights(s):
    import decode_step_kv_gb300 as fa
    c = s["case"]
    if c["int4"]:
        fa.fa_decode_int4(s["q"], s["k"], s["ks"], s["v"], s["vs"], s["table"], s["lens"], c["hq"], c["hkv"], c["d"],
                          s["scale"], s["window"], s["out"], acc=s["acc"], workspace=s["ws"])
    else:
        fa.fa_decode_weights(s["q"], s["k"], s["v"], None, s["table"], s["lens"], c["hq"], c["hkv"], c["d"],
                             s["scale"], s["window"], s["out"], s["acc"], workspace=s["ws"])
    return s["out"], s["acc"]


def own_evict(s):
    import decode_step_kv_gb300 as fa
    sink, recent = pins_of(s["case"])
    fa.fa_evict_kv(s["k"], s["v"], s["acc"], s["table"], s["lens"], s["new_lens"], budget=s["case"]["budget"],
                   n_sink=sink, n_recent=recent, kept=s["kept"])
    return s["k"], s["v"], s["acc"], s["kept"], s["new_lens"]


def row_index(s, t):
    """Cache row (in the flattened [.., head, token] order) of tokens t [B, n] of every KV head: [B, Hkv, n]."""
    hkv = s["case"]["hkv"]
    h = torch.arange(hkv, device=t.device).view(1, -1, 1)
    if s["table"] is None:
        b = torch.arange(t.shape[0], device=t.device).view(-1, 1, 1)
        return (b * hkv + h) * s["cap"] + t.unsqueeze(1)
    blk = torch.gather(s["table"].long(), 1, t // s["page"]).unsqueeze(1)
    return (blk * hkv + h) * s["page"] + (t % s["page"]).unsqueeze(1)


def plain_append(s):
    n = s["k_new"].shape[1]
    t = s["pos"].long().view(-1, 1) + torch.arange(n, device="cuda")
    at = row_index(s, t)
    for name in ("k", "v"):
        codes, scales = pack(s[name + "_new"].transpose(1, 2))
        s[name].flatten(0, 2)[at] = codes
        s[name + "s"].flatten(0, 2)[at] = scales
        back = unpack(s[name].flatten(0, 2)[at], s[name + "s"].flatten(0, 2)[at])
        s[name + "_out"].copy_(back.transpose(1, 2))
    return s["k_out"], s["v_out"]


def plain_attend(s):
    c = s["case"]
    b, hq, hkv, d, tq = c["batch"], c["hq"], c["hkv"], c["d"], c["tq"]
    cap = s["cap"]
    t = torch.arange(cap, device="cuda").expand(b, cap)
    at = row_index(s, t)

    def rows(name):
        x = s[name].flatten(0, 2)[at]
        return unpack(x, s[name + "s"].flatten(0, 2)[at]) if c["int4"] else x.float()

    # queries of one KV head: [B, Hkv, tq * G, D]
    q = s["q"].float().view(b, tq, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (q @ rows("k").transpose(2, 3)) * s["scale"]
    end = s["lens"].view(-1, 1) - tq + 1 + torch.arange(tq, device="cuda")                 # [B, tq]
    live = t.unsqueeze(1) < end.unsqueeze(2)
    if s["window"] is not None:
        w = s["window"].view(-1, 1, 1)
        live &= (w == 0) | (t.unsqueeze(1) >= end.unsqueeze(2) - w)
    live = live.unsqueeze(2).expand(b, tq, hq // hkv, cap).flatten(1, 2).unsqueeze(1)
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = p @ rows("v")
    s["out"].copy_(out.view(b, hkv, tq, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, tq, hq, d))
    if c["op"] != "weights":
        return s["out"]
    s["acc"].view(-1).index_add_(0, at.flatten(), p.sum(2).flatten())
    return s["out"], s["acc"]


def plain_evict(s):
    c = s["case"]
    budget, (sink, recent), cap = c["budget"], pins_of(c), s["cap"]
    b, hkv = c["batch"], c["hkv"]
    t = torch.arange(cap, device="cuda").expand(b, cap)
    at = row_index(s, t)
    n = s["lens"].long().view(-1, 1, 1)
    where = t.unsqueeze(1).expand(b, hkv, cap)
    acc = s["acc"].view(-1)[at]
    score = torch.where(torch.isnan(acc), torch.full_like(acc, -math.inf), acc)
    # largest total first, lowest index first among equals; then the pinned before the others, the absent last
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.ones_like(where)
    rank[(where < sink) | (where >= n - recent)] = 0
    rank[where >= n] = 2
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, stable=True).indices)[..., :budget]
    short = torch.arange(budget, device="cuda").expand(b, hkv, budget)
    keep = torch.where(n > budget, order.sort(-1).values, short)
    kept = torch.where(short < n, keep, torch.full_like(keep, -1))
    src = at.gather(-1, keep.clamp(max=cap - 1))
    dst = at[..., :budget]
    for name in ("k", "v"):
        flat = s[name].flatten(0, 2)
        flat[dst] = flat[src]
    s["acc"].view(-1)[at] = torch.where((where >= budget) & (where < n), torch.zeros_like(acc), acc)
    s["acc"].view(-1)[dst] = acc.gather(-1, keep.clamp(max=cap - 1))
    s["kept"].copy_(kept)
    s["new_lens"].copy_(s["lens"].clamp(max=budget))
    return s["k"], s["v"], s["acc"], s["kept"], s["new_lens"]


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        got = []
        for x in (s["k_new"], s["v_new"]):
            x = x.double()
            got.append(torch.empty_like(x))
            for j in range(0, case["d"], BLOCK):
                blk = x[..., j:j + BLOCK]
                scale = (blk.abs().max(dim=-1, keepdim=True).values / 7).half().double()
                code = torch.round(blk / torch.where(scale > 0, scale, torch.ones_like(scale)))
                got[-1][..., j:j + BLOCK] = code.clip(-7, 7) * scale
        return tuple(got)
    lens = lens_of(case)
    hkv, group, d, page = case["hkv"], case["hq"] // case["hkv"], case["d"], s["page"]

    def pages(x, b):
        """Sequence b's rows of a cache: [Hkv, cap, ...]."""
        if s["table"] is None:
            return x[b]
        return x[s["table"][b].long()].transpose(0, 1).flatten(1, 2)

    def value(name, b):
        x = pages(s[name], b)[:, :lens[b]]
        if not case["int4"]:
            return x.double()
        sc = pages(s[name + "s"], b)[:, :lens[b]].double()
        got = torch.empty(*x.shape[:-1], d, dtype=torch.float64, device=x.device)
        for e in range(d):                       # element e: its word, then its nibble
            j, o, n = e // 32, e % 32 // 8, e % 8
            byte = x[..., (o * (d // 32) + j) * 4 + n // 2].to(torch.int32)
            got[..., e] = ((byte >> (4 * (n % 2))) % 16 - 8).double() * sc[..., j]
        return got

    if case["op"] == "evict":
        k, v, acc = s["k"].clone(), s["v"].clone(), s["acc"].clone()
        kept = torch.full_like(s["kept"], -1)
        sink, recent = pins_of(case)
        for b, n in enumerate(lens):
            m = min(n, case["budget"])
            if n <= case["budget"]:
                kept[b, :, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
                continue
            a = pages(s["acc"], b)
            for h in range(hkv):
                mid = a[h, sink:n - recent]
                best = torch.argsort(mid, descending=True, stable=True)[:m - sink - recent].sort().values + sink
                pick = torch.cat([torch.arange(sink, device="cuda"), best, torch.arange(n - recent, n, device="cuda")])
                kept[b, h] = pick.int()
                for new, old in ((k, s["k"]), (v, s["v"]), (acc, s["acc"])):
                    if s["table"] is None:
                        new[b, h, :m] = old[b, h, pick]
                    else:
                        blk = s["table"][b].long()
                        to = torch.arange(m, device="cuda")
                        new[blk[to // page], h, to % page] = old[blk[pick // page], h, pick % page]
                gone = torch.arange(m, n, device="cuda")
                if s["table"] is None:
                    acc[b, h, gone] = 0
                else:
                    acc[s["table"][b].long()[gone // page], h, gone % page] = 0
        return k, v, acc, kept, torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if case["op"] == "weights" else None
    for b, n in enumerate(lens):
        k, v = value("k", b), value("v", b)
        w = case["window"] if b % 2 else 0
        for i in range(case["tq"]):
            end = n - case["tq"] + 1 + i
            if end <= 0:
                continue
            lo = max(0, end - w) if w else 0
            for h in range(hkv):
                q = s["q"][b, i, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ k[h, lo:end].T * s["scale"], dim=-1)
                out[b, i, h * group:(h + 1) * group] = p @ v[h, lo:end]
                if acc is None:
                    continue
                if s["table"] is None:
                    acc[b, h, lo:end] += p.sum(0)
                else:
                    t = torch.arange(lo, end, device="cuda")
                    acc[s["table"][b].long()[t // page], h, t % page] += p.sum(0)
    return out if acc is None else (out, acc)
