"""Cases of the step before attention over the cache, of attention of whole chunks, and of decode with sinks.

Four operators:
  * "rope":    rotary positions of one array of heads, with the RMS norm of each head in the same pass;
  * "append":  a projection's q, k and v rows: heads of q and k normed and rotated, q handed on, k and v
               written to the cache at each sequence's position;
  * "prefill": attention of a chunk of new tokens per sequence (a prompt, a part of one, or one token) over
               the cache, causal, with an optional sliding window and sinks;
  * "sinks":   decode attention with a sliding window and a few first tokens that stay visible.

``run`` computes them in elementary torch operations, or, with ``own``, by the package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
MOST_FLOPS = 2.3e12         # of a drawn chunk; the longest listed prompt has a little less
MOST_ROWS = 16384 * 48      # (token, head) rows of a drawn append or rotation


# --------------------------------------------------------------------------- cases
def listed():
    def case(name, op, batch, hq, hkv, d, lo, hi, **more):
        c = {"name": name, "op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
             "lo": lo, "hi": hi,            # tokens in each sequence's cache after the call, spread from hi to lo
             "nlo": 1, "nhi": 1,            # new tokens of each sequence, spread from nhi to nlo
             "paged": True, "page": 16, "window": 0, "sink": 0, "tq": 1, "int8": False,
             "dtype": "fp16", "rot": d, "inter": False, "norm": True, "base": 10000.0,
             "scaling": "none", "factor": 1.0, "orig": 8192}
        c.update(more)
        return c

    return [
        # the queries of one decode step of 64 sequences: a call that is all latency
        case("rope_64x1_d128", "rope", 64, 32, 8, 128, 1, 8192),
        # a prompt's queries, a quarter of the head rotated in interleaved pairs, positions scaled by parts
        case("rope_8x2048_d256_part", "rope", 8, 16, 8, 256, 2048, 40000, nlo=2048, nhi=2048, dtype="bf16",
             rot=64, inter=True, base=500000.0, scaling="yarn", factor=8.0),
        # one decode step's q, k and v of 64 sequences
        case("append_64x1_d128", "append", 64, 32, 8, 128, 1, 8192),
        # a batch of prompts of odd lengths, G = 8
        case("append_5x1k-5k_d128_bf16", "append", 5, 64, 8, 128, 1021, 5003, nlo=1021, nhi=5003, dtype="bf16",
             base=500000.0),
        # a chunk far into a long document, scaled positions, no norm, 32-bit projections
        case("append_1x2048_at_126k_d256", "append", 1, 16, 8, 256, 131072, 131072, nlo=2048, nhi=2048,
             dtype="fp32", norm=False, scaling="linear", factor=16.0, paged=False),
        # the last part of a short chat's prompt
        case("prefill_1x64_of_512_d128", "prefill", 1, 8, 2, 128, 512, 512, nlo=64, nhi=64),
        # parts of prompts of odd sizes beside single decode tokens, sliding windows with sinks on odd sequences
        case("prefill_16x1-700_of_16k_d128", "prefill", 16, 32, 4, 128, 5003, 16381, nlo=1, nhi=701, window=4096,
             sink=4),
        # prompts of mixed length at once, head_dim 256
        case("prefill_4x1k-8k_d256", "prefill", 4, 16, 8, 256, 1024, 8192, nlo=1024, nhi=8192, paged=False),
        # one chunk over a long document: few rows, a long axis of keys
        case("prefill_1x512_of_128k_d128", "prefill", 1, 32, 8, 128, 131072, 131072, nlo=512, nhi=512),
        # a whole long prompt
        case("prefill_1x16k_d128", "prefill", 1, 32, 8, 128, 16384, 16384, nlo=16384, nhi=16384, page=64),
        # one chat beyond its window
        case("sinks_1x2k_d128", "sinks", 1, 8, 2, 128, 2048, 2048, paged=False, window=1000, sink=4),
        # a served batch of long chats, drafts of 3 tokens verified at once, int8 V
        case("sinks_32x1k-32k_d128_3q_int8", "sinks", 32, 32, 8, 128, 1021, 32768, window=8192, sink=20, tq=3,
             int8=True),
    ]


def draw(rng):
    def spread(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["rope", "append", "prefill", "prefill", "sinks"])
    d = rng.choice([128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    c = {"op": op, "d": d, "hkv": hkv, "hq": hq, "paged": rng.random() < 0.7, "page": rng.choice([16, 16, 32, 48, 128]),
         "window": 0, "sink": 0, "tq": 1, "int8": False, "dtype": rng.choice(["fp16", "bf16", "fp32"]),
         "rot": rng.choice([d, d, d // 2, d // 4, 16 * rng.randint(1, d // 16)]), "inter": rng.random() < 0.4,
         "norm": rng.random() < 0.6, "base": rng.choice([10000.0, 500000.0]),
         "scaling": rng.choice(["none", "none", "linear", "ntk", "yarn"]), "factor": 1.0, "orig": 8192,
         "nlo": 1, "nhi": 1}
    if c["scaling"] != "none":
        c["factor"] = rng.choice([2.0, 8.0, 13.0])
    if op == "sinks":
        c["batch"] = spread(1, 48)
        c["hi"] = spread(64, min(65536, (1 << 20) // (c["batch"] * (d // 128))))
        c["window"] = spread(16, c["hi"])
        c["sink"] = rng.choice([1, 4, 4, 16, 61])
        c["tq"] = rng.choice([1, 1, 1, 2, 4])
        c["int8"] = rng.random() < 0.4
    elif op == "prefill":
        while True:
            c["batch"] = spread(1, 32)
            c["nhi"] = spread(1, 8192)
            c["nlo"] = max(1, int(c["nhi"] * rng.choice([1.0, 0.5, 0.05])))
            c["hi"] = min(65536, c["nhi"] + rng.choice([0, spread(1, 65536)]))
            c["lo"] = max(c["nhi"], int(c["hi"] * rng.choice([1.0, 0.3])))
            c["window"], c["sink"] = rng.choice([(0, 0), (0, 0), (spread(16, c["hi"]), 0),
                                                 (spread(16, c["hi"]), rng.choice([1, 4, 130]))])
            # products of whole rectangles, which is what the plain form computes
            if c["batch"] * c["nhi"] * c["hi"] * c["hq"] * 4 * d <= MOST_FLOPS and \
                    c["batch"] * c["hi"] * hkv * d <= 1 << 30:
                break
    else:
        while True:
            c["batch"] = spread(1, 64)
            c["nhi"] = spread(1, 16384)
            if c["batch"] * c["nhi"] * (hq + 2 * hkv) <= MOST_ROWS:
                break
        c["nlo"] = max(1, int(c["nhi"] * rng.choice([1.0, 0.5, 0.05])))
        c["hi"] = c["nhi"] + rng.choice([0, spread(1, 20000)])
    c.setdefault("lo", max(c["nhi"], int(c["hi"] * rng.choice([1.0, 0.5, 0.05]))))
    return c


def spread_of(case, lo, hi):
    n = case["batch"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def lens_of(case):
    """Tokens of each sequence after the call, its new ones among them."""
    return [max(n, m) for n, m in zip(spread_of(case, case["lo"], case["hi"]), news_of(case))]


def news_of(case):
    return spread_of(case, case["nlo"], case["nhi"])


def windows_of(case):
    """A sliding window on odd sequences (on every one where sinks are the point)."""
    return [case["window"] if b % 2 or case["op"] == "sinks" else 0 for b in range(case["batch"])]


def seen(at, window, sink):
    """Keys that the token at position ``at`` sees."""
    if not window or at < window:
        return at + 1
    return window + min(sink, at + 1 - window)


def work(case):
    hq, hkv, d, g = case["hq"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    new = sum(news_of(case))
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        return {"bytes": new * hq * d * (size + (2 if size == 4 else size)), "flops": new * hq * d * 7}
    if case["op"] == "append":
        return {"bytes": new * (hq + 2 * hkv) * d * (size + 2), "flops": new * (hq + hkv) * d * 7}
    keys = pairs = 0
    for n, m, w in zip(lens_of(case), news_of(case), windows_of(case)):
        m = case["tq"] if case["op"] == "sinks" else m
        first, last = max(0, n - m), n - 1
        lo = max(0, first - w + 1) if w else 0
        keys += last + 1 - lo + min(case["sink"], lo)
        if not w:
            pairs += (first + 1 + last + 1) * (last - first + 1) // 2
        else:
            pairs += sum(seen(at, w, case["sink"]) for at in range(first, last + 1))
    rows = new * case["tq"] * hq * d
    v = d + d // 16 if case["int8"] else 2 * d
    return {"bytes": keys * hkv * (2 * d + v) + rows * 4, "flops": pairs * hkv * g * 4 * d}


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    b, hq, hkv, d, op = case["batch"], case["hq"], case["hkv"], case["d"], case["op"]
    lens, new = lens_of(case), news_of(case)
    s = {"case": case, "scale": d ** -0.5}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"] = ints(starts)
    s["lens"] = ints(lens)
    s["positions"] = ints([n - m for n, m in zip(lens, new)])
    if op in ("rope", "append"):
        dt = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]
        heads = hq if op == "rope" else hq + 2 * hkv
        # one projection's output, its q, k and v side by side in every token's row; channels of unlike size
        x = torch.empty(starts[-1], heads, d, dtype=dt, device=dev).normal_(generator=g)
        x *= torch.rand(heads, d, generator=g, device=dev).add_(0.5).to(dt)
        s["q"] = x[:, :hq]
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = torch.rand(d, generator=g, device=dev).add_(0.5).to(dt)
            s["kw"] = torch.rand(d, generator=g, device=dev).add_(0.5).to(dt)
        s["q_out"] = torch.zeros(starts[-1], hq, d, dtype=dt if op == "rope" and dt != torch.float32
                                 else torch.float16, device=dev)
        if op == "rope":
            s["at"] = torch.cat([torch.arange(n - m, n, dtype=torch.int32) for n, m in zip(lens, new)]).to(dev)
        else:
            s["k"], s["v"] = x[:, hq:hq + hkv], x[:, hq + hkv:]
        if own:
            import decode_step_kv_gb300 as fa
            s["table"], s["magnitude"] = fa.fa_rope_table(
                case["rot"], case["base"], scaling=None if case["scaling"] == "none" else case["scaling"],
                factor=case["factor"], original_len=case["orig"], device=dev)
        if op == "rope":
            return s
    page = case["page"] if case["paged"] else 16
    blocks = -(-max(lens) // page)
    s["page"], s["cap"] = page, blocks * page
    if case["paged"]:
        total = b * blocks + 3
        order = torch.randperm(total, generator=g, device=dev)[:b * blocks]
        s["blocks"] = order.to(torch.int32).view(b, blocks).contiguous()
        shape = (total, hkv, page)
    else:
        s["blocks"] = None
        shape = (b, hkv, s["cap"])
    for n in ("kc", "vc"):
        s[n] = torch.empty(*shape, d, dtype=torch.float16, device=dev)
        if op == "append":
            s[n].zero_()
        else:
            s[n].normal_(generator=g)
    if op == "append":
        return s
    s["vs"] = None
    if case["int8"]:
        blk = s["vc"].float().unflatten(-1, (d // 32, 32))
        s["vs"] = (blk.abs().amax(-1) / 127.0).half()
        s["vc"] = torch.round(blk / s["vs"].float().unsqueeze(-1)).clamp_(-127, 127).flatten(-2).to(torch.int8)
    s["window"] = ints(windows_of(case)) if case["window"] else None
    rows = (b, case["tq"]) if op == "sinks" else (starts[-1],)
    s["q"] = torch.empty(*rows, hq, d, dtype=torch.float16, device=dev).normal_(generator=g)
    s["out"] = torch.empty(*rows, hq, d, dtype=torch.float16, device=dev)
    if own:
        import decode_step_kv_gb300 as fa
        if op == "sinks":
            s["ws"] = fa.alloc_workspace_sinks(b, case["tq"], hq, hkv, d, s["cap"])
        else:
            s["ws"] = fa.alloc_workspace_prefill(b, starts[-1], hq, hkv, d, s["cap"])
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": own_rope, "append": own_append, "prefill": own_prefill, "sinks": own_sinks}[op](state)
    return {"rope": plain_rope, "append": plain_append, "prefill": plain_prefill, "sinks": plain_sinks}[op](state)


def own_rope(s):
    import decode_step_kv_gb300 as fa
    fa.fa_rope(s["q"], s["at"], s["table"], s["q_out"], weight=s["qw"], eps=EPS, interleaved=s["case"]["inter"],
               magnitude=s["magnitude"])
    return s["q_out"]


def own_append(s):
    import decode_step_kv_gb300 as fa
    fa.fa_rope_append_kv(s["q"], s["k"], s["v"], s["q_out"], s["kc"], s["vc"], None, s["blocks"], s["starts"],
                         s["positions"], s["table"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                         interleaved=s["case"]["inter"], magnitude=s["magnitude"])
    return s["q_out"], s["kc"], s["vc"]


def own_prefill(s):
    import decode_step_kv_gb300 as fa
    c = s["case"]
    fa.fa_prefill(s["q"], s["kc"], s["vc"], s["vs"], s["blocks"], s["starts"], s["lens"], c["hq"], c["hkv"], c["d"],
                  s["scale"], s["window"], s["out"], n_sink=c["sink"], workspace=s["ws"])
    return s["out"]


def own_sinks(s):
    import decode_step_kv_gb300 as fa
    c = s["case"]
    fa.fa_decode_sinks(s["q"], s["kc"], s["vc"], s["vs"], s["blocks"], s["lens"], c["hq"], c["hkv"], c["d"],
                       s["scale"], s["window"], s["out"], n_sink=c["sink"], workspace=s["ws"])
    return s["out"]


def rates(case):
    """Radians per position of every pair, in 64 bits, and the factor on cos and sin."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    r = base ** (torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / -rot)
    if case["scaling"] == "linear":
        r = r / f
    if case["scaling"] != "yarn":
        return r, 1.0
    # pairs that turn more than 32 times within the original length keep their rate, those that turn
    # less than once are slowed by the factor, a ramp between them

    def pair(turns):
        return rot * math.log(case["orig"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    first, last = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
    ramp = (torch.arange(rot // 2, dtype=torch.float64, device="cuda") - first) / max(last - first, 0.001)
    ramp = ramp.clamp(0, 1)
    return r * (1 - ramp) + r / f * ramp, 0.1 * math.log(f) + 1.0


def turn(case, x, at, weight):
    """Rows x [N, H, D] normed and rotated to positions at [N], in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r, m = rates(case)
    angle = at.double().unsqueeze(-1) * r
    cos, sin = (torch.cos(angle) * m).float().unsqueeze(1), (torch.sin(angle) * m).float().unsqueeze(1)
    rot = case["rot"]
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def plain_rope(s):
    s["q_out"].copy_(turn(s["case"], s["q"], s["at"], s["qw"]))
    return s["q_out"]


def tokens_of(s):
    """Sequence and cache position of every new token."""
    starts = s["starts"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, s["positions"].long()[b] + t - starts[b]


def plain_append(s):
    c = s["case"]
    b, at = tokens_of(s)
    s["q_out"].copy_(turn(c, s["q"], at, s["qw"]))
    k, v = turn(c, s["k"], at, s["kw"]).half(), s["v"].half()
    if s["blocks"] is None:
        s["kc"][b, :, at] = k
        s["vc"][b, :, at] = v
    else:
        blk = s["blocks"].long()[b, at // s["page"]]
        s["kc"][blk, :, at % s["page"]] = k
        s["vc"][blk, :, at % s["page"]] = v
    return s["q_out"], s["kc"], s["vc"]


def rows_of(s, b):
    """Sequence b's K and V in 32 bits: [Hkv, cap, D] each."""
    got = []
    for name in ("kc", "vc"):
        x = s[name][b] if s["blocks"] is None else s[name][s["blocks"][b].long()].transpose(0, 1).flatten(1, 2)
        x = x.float()
        if name == "vc" and s["vs"] is not None:
            z = s["vs"][b] if s["blocks"] is None else s["vs"][s["blocks"][b].long()].transpose(0, 1).flatten(1, 2)
            x = (x.unflatten(-1, (-1, 32)) * z.float().unsqueeze(-1)).flatten(-2)
        got.append(x)
    return got


def attend(c, q, k, v, at, scale, window):
    """q [N, Hq, D] at positions at [N] over one sequence's k and v [Hkv, cap, D]."""
    hkv, g = c["hkv"], c["hq"] // c["hkv"]
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    t = torch.arange(k.shape[1], device=q.device)
    at = at.view(-1, 1)
    live = t <= at
    if window:
        live &= (t > at - window) | (t < c["sink"])
    for h in range(hkv):
        for lo in range(0, q.shape[0], 4096):
            x = q[lo:lo + 4096, h * g:(h + 1) * g].float().transpose(0, 1)          # [G, n, D]
            score = (x @ k[h].T) * scale
            score.masked_fill_(~live[lo:lo + 4096], -math.inf)
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
            total = p.sum(-1, keepdim=True)
            y = (p @ v[h]) / torch.where(total > 0, total, torch.ones_like(total))
            out[lo:lo + 4096, h * g:(h + 1) * g] = y.transpose(0, 1)
    return out


def plain_prefill(s):
    c = s["case"]
    start = 0
    for b, (n, m, w) in enumerate(zip(lens_of(c), news_of(c), windows_of(c))):
        k, v = (x[:, :n] for x in rows_of(s, b))
        at = torch.arange(n - m, n, device="cuda")
        s["out"][start:start + m] = attend(c, s["q"][start:start + m], k, v, at, s["scale"], w)
        start += m
    return s["out"]


def plain_sinks(s):
    c = s["case"]
    for b, (n, w) in enumerate(zip(lens_of(c), windows_of(c))):
        k, v = (x[:, :n] for x in rows_of(s, b))
        at = torch.arange(n - c["tq"], n, device="cuda")
        s["out"][b] = attend(c, s["q"][b], k, v, at, s["scale"], w)
    return s["out"]


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d, rot, hkv, g = case["d"], case["rot"], case["hkv"], case["hq"] // case["hkv"]
    lens, new = lens_of(case), news_of(case)
    if case["op"] in ("rope", "append"):
        base, f = case["base"], case["factor"]
        if case["scaling"] == "ntk" and rot > 2:
            base *= f ** (rot / (rot - 2.0))
        rate, size = [], 1.0
        for j in range(rot // 2):
            r = math.exp(-2.0 * j / rot * math.log(base))
            if case["scaling"] == "linear":
                r /= f
            elif case["scaling"] == "yarn":
                size = 1.0 + math.log(f) / 10.0
                edge = [rot / 2.0 * math.log(case["orig"] / (2.0 * math.pi * n)) / math.log(base) for n in (32, 1)]
                lo, hi = max(0, math.floor(edge[0])), min(rot - 1, math.ceil(edge[1]))
                slow = min(1.0, max(0.0, (j - lo) / (hi - lo if hi > lo else 0.001)))
                r = (1.0 - slow) * r + slow * r / f
            rate.append(r)
        at = torch.cat([torch.arange(n - m, n, device="cuda", dtype=torch.float64) for n, m in zip(lens, new)])
        z = torch.polar(torch.full((rot // 2, 1), size, dtype=torch.float64, device="cuda"),
                        torch.tensor(rate, dtype=torch.float64, device="cuda").view(-1, 1) * at).T    # [N, rot / 2]

        def value(x, weight):
            y = x.double()
            if weight is not None:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + EPS) * weight.double()
            ends = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
            turned = torch.complex(y[..., ends[0]].contiguous(), y[..., ends[1]].contiguous()) * z.unsqueeze(1)
            y[..., ends[0]], y[..., ends[1]] = turned.real, turned.imag
            return y

        q = value(s["q"], s["qw"])
        if case["op"] == "rope":
            return q
        caches = []
        for x, cache in ((value(s["k"], s["kw"]), s["kc"]), (s["v"].double(), s["vc"])):
            to = cache.double()
            row = 0
            for b, (n, m) in enumerate(zip(lens, new)):
                if s["blocks"] is None:
                    to[b, :, n - m:n] = x[row:row + m].transpose(0, 1)
                else:
                    t = torch.arange(n - m, n, device="cuda")
                    to[s["blocks"][b].long()[t // s["page"]], :, t % s["page"]] = x[row:row + m]
                row += m
            caches.append(to)
        return (q, *caches)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    flat, q = out.view(-1, case["hq"], d), s["q"].view(-1, case["hq"], d)
    row = 0
    for b, (n, m, w) in enumerate(zip(lens, new, windows_of(case))):
        m = case["tq"] if case["op"] == "sinks" else m
        full = []
        for name in ("kc", "vc"):
            x = s[name][b] if s["blocks"] is None else torch.cat(list(s[name][s["blocks"][b].long()]), dim=1)
            x = x[:, :n].double()
            if name == "vc" and case["int8"]:
                y = s["vs"][b] if s["blocks"] is None else torch.cat(list(s["vs"][s["blocks"][b].long()]), dim=1)
                x = x * torch.repeat_interleave(y[:, :n].double(), 32, dim=-1)
            full.append(x)
        for i in range(0, m, 1024):
            j = min(m, i + 1024)
            if n - m + j <= 0:
                continue
            # the block's first row begins at lo, its last ends at hi
            lo, hi = (max(0, n - m + i - w + 1) if w else 0), n - m + j
            t = torch.arange(lo, hi, device="cuda")
            if w and case["sink"] and lo:
                t = torch.cat([torch.arange(min(case["sink"], lo), device="cuda"), t])
            at = torch.arange(n - m + i, n - m + j, device="cuda").view(-1, 1)
            hide = t > at
            if w:
                hide |= (t <= at - w) & (t >= case["sink"])
            for h in range(hkv):
                x = q[row + i:row + j, h * g:(h + 1) * g].double().transpose(0, 1)
                p = (x @ full[0][h][t].T * s["scale"]).masked_fill(hide, -math.inf)
                p = torch.softmax(p, dim=-1).nan_to_num(0.0)
                flat[row + i:row + j, h * g:(h + 1) * g] = (p @ full[1][h][t]).transpose(0, 1)
        row += m
    return out
