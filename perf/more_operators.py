"""The operators of a decode step over a latent cache held in 8 bits, each in its
plain form and as the library's call, over the sizes they are used at.

  latent_cache_write_fp8              normalized and rotated latent rows, quantized into the paged cache
  latent_cache_read_fp8               rows of the quantized cache, read back in order as bf16
  paged_latent_attention_fp8          one new token per request over the quantized cache
  shared_prefix_latent_attention_fp8  the same for a batch whose requests begin with the same tokens

A cached row is one fp32 scale times (K e4m3 codes | P bf16 numbers), the
position columns divided by the latent's scale, so that one factor serves all.

run(state) makes one pass: elementary torch operations in fp32 (rotary angles
in fp64) where `own` is false, the library's entry point where it is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TOP = 448.0                  # the largest e4m3 value
LEAST = 2.0 ** -60           # the smallest scale of a row


# ------------------------------------------------------------------- cases

def listed():
    return [
        # Decode batch: the normalized latent of the pre-projection and the 64 position columns of its row, three padded rows.
        {"name": "write decode 32", "op": "write", "M": 32, "K": 512, "P": 64, "norm": 0, "layout": "interleaved",
         "page": 64, "maxpos": 16384, "pad": 3},
        # Prompt: raw latents, normalized on the way into the cache, a few padded rows.
        {"name": "write prompt 8191", "op": "write", "M": 8191, "K": 512, "P": 64, "norm": 1, "layout": "interleaved",
         "page": 64, "maxpos": 131072, "pad": 17},
        # A chunk of a prompt: the tokens before it of a few chats, read back for the attention of its own.
        {"name": "read 5 up to 2000", "op": "read", "B": 5, "K": 512, "P": 64, "page": 64, "maxlen": 2000, "even": 0,
         "pad": 7, "later": 0, "shape": 1},
        # Long documents continued in chunks: a window of each, from an odd token on, small pages.
        {"name": "read 3 x 40001", "op": "read", "B": 3, "K": 512, "P": 64, "page": 16, "maxlen": 40001, "even": 1,
         "pad": 0, "later": 1, "shape": 2},
        # One request of a chat, all 128 heads: the latency of a single decode.
        {"name": "attention 1 x 701", "op": "attention", "B": 1, "H": 128, "K": 512, "P": 64, "DV": 512, "page": 64,
         "maxlen": 701, "even": 1, "empty": 0, "shape": 3},
        # Two long documents with a sixteenth of the heads on this GPU, small pages: split over the length.
        {"name": "attention 2 x 131071", "op": "attention", "B": 2, "H": 16, "K": 512, "P": 64, "DV": 512, "page": 32,
         "maxlen": 131071, "even": 1, "empty": 0, "shape": 4},
        # Large even batch, 48 heads as wide as the latent, no position columns apart: the most bytes.
        {"name": "attention 128 x 8000", "op": "attention", "B": 128, "H": 48, "K": 512, "P": 0, "DV": 512, "page": 16,
         "maxlen": 8000, "even": 1, "empty": 0, "shape": 5},
        # Large batch, all heads, lengths from a few tokens to a long context, a padded (empty) row in it.
        {"name": "attention 96 mixed", "op": "attention", "B": 96, "H": 128, "K": 512, "P": 64, "DV": 512, "page": 64,
         "maxlen": 32768, "even": 0, "empty": 1, "shape": 6},
        # Four samples of one question: a short prompt in common, their own few tokens behind it, all heads.
        {"name": "shared 4 x 900 + 60", "op": "shared", "B": 4, "H": 128, "K": 512, "P": 64, "DV": 512, "page": 64,
         "prefix": 900, "maxlen": 60, "even": 0, "empty": 1, "shape": 7},
        # Requests about one long document, a sixteenth of the heads on this GPU.
        {"name": "shared 64 x 32769 + 1000", "op": "shared", "B": 64, "H": 16, "K": 512, "P": 64, "DV": 512, "page": 64,
         "prefix": 32769, "maxlen": 1000, "even": 0, "empty": 1, "shape": 8},
        # A serving batch behind one system prompt, 48 heads, an odd number of them, uneven conversations.
        {"name": "shared 131 x 3001 + 4096", "op": "shared", "B": 131, "H": 48, "K": 512, "P": 0, "DV": 512, "page": 16,
         "prefix": 3001, "maxlen": 4096, "even": 0, "empty": 3, "shape": 9},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "shared", "shared"])
    if op == "write":
        K, P = rng.choice([(512, 64), (512, 64), (512, 0), (256, 64)])
        M = _log(rng, 1, 8000)
        return {"op": op, "M": M, "K": K, "P": P, "norm": rng.randrange(2), "layout": rng.choice(["interleaved", "half"]),
                "page": rng.choice([16, 32, 64, 128]), "maxpos": _log(rng, 100, 2000000), "pad": rng.randrange(0, min(M, 9))}
    if op == "read":
        K, P = rng.choice([(512, 64), (512, 64), (512, 0), (256, 64)])
        B = _log(rng, 1, 60)
        return {"op": op, "B": B, "K": K, "P": P, "page": rng.choice([8, 16, 32, 48, 64, 128]),
                "maxlen": _log(rng, 1, min(40000, 120000 // B)), "even": rng.randrange(2), "pad": rng.randrange(0, 9),
                "later": rng.randrange(2), "shape": rng.randrange(1 << 20)}
    K, P, DV = rng.choice([(512, 64, 512), (512, 64, 512), (512, 0, 512), (256, 64, 256)])
    heads = rng.choice([1, 8, 16, 24, 48, 64, 100, 128])
    page = rng.choice([8, 16, 32, 48, 64, 128, 256])
    if op == "attention":
        B = _log(rng, 1, 96)
        return {"op": op, "B": B, "H": heads, "K": K, "P": P, "DV": DV, "page": page, "maxlen": _log(rng, 1, min(100000, 400000 // B)),
                "even": rng.randrange(2), "empty": rng.randrange(0, 1 + B // 8), "shape": rng.randrange(1 << 20)}
    B = _log(rng, 2, 96)
    return {"op": op, "B": B, "H": heads, "K": K, "P": P, "DV": DV, "page": page, "prefix": _log(rng, 100, min(32768, 8000000 // (B * heads))),
            "maxlen": _log(rng, 1, min(4096, 200000 // B)), "even": rng.randrange(2), "empty": rng.randrange(0, 1 + B // 8),
            "shape": rng.randrange(1 << 20)}


def _lens(c):
    """Request lengths (behind the prefix, where there is one)."""
    r = random.Random(c["shape"])
    lens = [c["maxlen"] if c["even"] else _log(r, 1, c["maxlen"]) for _ in range(c["B"])]
    for i in range(c.get("empty", 0)):
        lens[(7 * i + 3) % c["B"]] = 0
    return lens


def _firsts(c):
    """First token to be read of each request."""
    r = random.Random(c["shape"] + 1)
    return [r.randrange(0, 1 + n // 3) if c["later"] else 0 for n in _lens(c)]


def work(case):
    c = case
    row = c["K"] + 2 * c["P"] + 4                        # codes, position columns, scale
    if c["op"] == "write":
        live, W = c["M"] - c["pad"], c["K"] + c["P"]
        return {"bytes": 2 * live * W + live * row + 8 * c["M"] + 8 * live + 4 * 64 + 2 * c["K"] * c["norm"],
                "flops": live * (4 * c["K"] * c["norm"] + 2 * c["K"] + 3 * 64)}
    lens = _lens(c)
    if c["op"] == "read":
        lens = [n - f for n, f in zip(lens, _firsts(c))]
        total = sum(lens)
        return {"bytes": total * (row + 2 * (c["K"] + c["P"])) + 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["B"],
                "flops": total * (c["K"] + c["P"])}
    DK, total, held = c["K"] + c["P"], sum(lens), sum(lens)
    pages = sum(-(-n // c["page"]) for n in lens)
    if c["op"] == "shared":
        total += c["B"] * c["prefix"]
        held += c["prefix"]
        pages += -(-c["prefix"] // c["page"])
    return {"bytes": held * row + 4 * pages + 2 * c["B"] * c["H"] * (DK + c["DV"]) + 4 * c["B"] * (c["H"] + 1),
            "flops": 2 * total * c["H"] * (DK + c["DV"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _tables(g, held, width, spare):
    """Block tables [len(held), width] over shuffled pages, and how many pages there are."""
    pages = sum(held) + spare
    pool = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    mine = torch.arange(width, device=DEV)[None] < torch.tensor(held, device=DEV)[:, None]
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=DEV)
    table[mine] = pool[:sum(held)]
    return table, pages


def _cache(g, pages, page, K, P):
    """(cache, scales): rows as a serving loop has them, normalized latents with a weight and rotated position columns."""
    gamma = torch.rand(K, generator=g, device=DEV) + 0.5
    cache = torch.empty(pages, page, K + 2 * P, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, page, dtype=torch.float32, device=DEV)
    at = max(1, (1 << 28) // (page * K))                 # so many pages at a time
    for i in range(0, pages, at):
        x = torch.randn(min(at, pages - i), page, K, generator=g, device=DEV).mul_(gamma)
        s = (x.abs().amax(-1) / TOP).clamp(min=LEAST)
        scales[i:i + at] = s
        cache[i:i + at, :, :K] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if P:
            pe = torch.randn(x.shape[0], page, P, generator=g, device=DEV) / s[..., None]
            cache[i:i + at, :, K:] = pe.bfloat16().view(torch.uint8)
    return cache, scales


def prepare(case, seed):
    """Inputs, and the output buffers that a decode loop keeps from step to step."""
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    K, P, page = c["K"], c["P"], c["page"]
    if c["op"] == "write":
        M = c["M"]
        first = torch.randint(0, c["maxpos"], (1,), generator=g, device=DEV)
        spread = torch.randint(0, c["maxpos"], (M,), generator=g, device=DEV)
        run = (first + torch.arange(M, device=DEV)) % c["maxpos"]
        row = _randn(g, M, 1536 + K + P)                 # the fused projection's row: q latent, kv latent, position columns
        pages = -(-M // page) + 4
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:M]
        if c["pad"]:
            slots[M - c["pad"]:] = -1
        cache, scales = _cache(g, pages, page, K, P)
        s.update(kv=row[:, 1536:1536 + K], pe=row[:, 1536 + K:] if P else None, slots=slots, positions=spread if M < 512 else run,
                 inv_freq=10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=DEV) / 64),
                 gamma=(torch.rand(K, generator=g, device=DEV) + 0.5).to(torch.bfloat16) if c["norm"] else None,
                 cache=cache, scales=scales, off=K + P - 64)
        return s
    lens = _lens(c)
    held = [-(-n // page) for n in lens]
    width = max(max(held), 1) + 1
    if c["op"] == "read":
        table, pages = _tables(g, held, width, 4)
        s["cache"], s["scales"] = _cache(g, pages, page, K, P)
        first = _firsts(c)
        starts = [0]
        for n, f in zip(lens, first):
            starts.append(starts[-1] + n - f)
        s.update(table=table, starts=torch.tensor(starts, dtype=torch.int32, device=DEV), rows=starts[-1] + c["pad"],
                 first=torch.tensor(first, dtype=torch.int32, device=DEV) if c["later"] else None,
                 out=_randn(g, starts[-1] + c["pad"], K + P))
        return s
    before = -(-c["prefix"] // page) if c["op"] == "shared" else 0
    table, pages = _tables(g, held + [before], max(width, before), 4)
    if before:
        s.update(prefix_table=table[-1, :before].contiguous(), prefix_len=torch.tensor([c["prefix"]], dtype=torch.int32, device=DEV))
    s["cache"], s["scales"] = _cache(g, pages, page, K, P)
    s.update(q=_randn(g, c["B"], c["H"], K + P), table=table[:-1, :width].contiguous(),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scale=((K + P) / 3.0) ** -0.5,
             out=torch.empty(c["B"], c["H"], c["DV"], dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(c["B"], c["H"], dtype=torch.float32, device=DEV))
    return s


# ------------------------------------------------------------- plain forms

def _views(s):
    """The cache as the values it holds: codes, position columns and scales."""
    K = s["c"]["K"]
    return s["cache"][..., :K].view(torch.float8_e4m3fn), s["cache"][..., K:].view(torch.bfloat16), s["scales"]


def _plain_write(s):
    c, cache, K = s["c"], s["cache"], s["c"]["K"]
    x = s["kv"].float()
    if c["norm"]:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["gamma"].float()
    if s["pe"] is not None:
        x = torch.cat([x, s["pe"].float()], -1)
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin, v = angle.cos().float(), angle.sin().float(), x[:, s["off"]:]
    if c["layout"] == "half":
        a, b = v.chunk(2, -1)
        v = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = v[:, 0::2], v[:, 1::2]
        v = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    x = torch.cat([x[:, :s["off"]], v], -1)
    scale = (x[:, :K].abs().amax(-1) / TOP).clamp(min=LEAST)
    x = x / scale[:, None]
    row = torch.cat([x[:, :K].clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8), x[:, K:].bfloat16().view(torch.uint8)], -1)
    # Rows without a slot land on row 0 of a copy that is one row longer.
    at = torch.where(s["slots"] >= 0, s["slots"], s["scales"].numel())
    for flat, new in ((cache.view(-1, cache.shape[-1]), row), (s["scales"].view(-1), scale)):
        longer = torch.cat([flat, flat[:1]])
        longer[at] = new
        flat.copy_(longer[:-1])
    return _views(s)


def _rows(s, entries, at):
    """Rows of the tokens `at` on the pages `entries`, in fp32."""
    page, K = s["c"]["page"], s["c"]["K"]
    flat = entries.long().clamp(min=0) * page + at % page
    row = s["cache"].view(-1, s["cache"].shape[-1])[flat]
    x = torch.cat([row[..., :K].view(torch.float8_e4m3fn).float(), row[..., K:].contiguous().view(torch.bfloat16).float()], -1)
    return x * s["scales"].view(-1)[flat][..., None]


def _plain_read(s):
    c, starts, B = s["c"], s["starts"].long(), s["c"]["B"]
    r = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(starts[1:], r, right=True).clamp(max=B - 1)
    at = r - starts[b] + (0 if s["first"] is None else s["first"][b])
    live = r < starts[B]
    at = torch.where(live, at, 0)
    x = _rows(s, s["table"][b, at // c["page"]], at)
    s["out"].copy_(torch.where(live[:, None], x.bfloat16(), s["out"]))
    return s["out"]


def _plain_attention(s):
    c, q, lens = s["c"], s["q"].float(), s["lens"]
    B, H, DV = c["B"], c["H"], c["DV"]
    at = torch.arange(s["table"].shape[1] * c["page"], device=DEV)
    valid = at[None] < lens[:, None]
    k = torch.where(valid[..., None], _rows(s, s["table"][:, at // c["page"]], at), 0.0)
    score = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    score = torch.where(valid[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    if c["op"] == "shared":
        at = torch.arange(c["prefix"], device=DEV)
        front = _rows(s, s["prefix_table"][at // c["page"]], at)
        first = torch.matmul(q.view(B * H, -1), front.T).view(B, H, -1) * s["scale"]
        top = torch.maximum(top, first.amax(-1, keepdim=True))
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total, out = p.sum(-1, keepdim=True), torch.matmul(p, k[..., :DV])
    if c["op"] == "shared":
        p = torch.exp(first - top)
        total = total + p.sum(-1, keepdim=True)
        out = out + torch.matmul(p.view(B * H, -1), front[:, :DV]).view(B, H, DV)
    out = out / torch.where(total > 0, total, 1.0)
    return out.bfloat16(), (top + torch.log(total))[..., 0]


_PLAIN = {"write": _plain_write, "read": _plain_read, "attention": _plain_attention, "shared": _plain_attention}


# ------------------------------------------------------- the library's calls

def _own(s):
    import gemm_dsnq_dual_gb300 as dsnq
    c = s["c"]
    if c["op"] == "write":
        dsnq.latent_cache_write_fp8(s["kv"], s["pe"], s["positions"], s["slots"], s["inv_freq"], s["cache"], s["scales"], gamma=s["gamma"],
                                    eps=EPS, normalize=bool(c["norm"]), rope_offset=s["off"], layout=c["layout"])
        return _views(s)
    if c["op"] == "read":
        return dsnq.latent_cache_read_fp8(s["cache"], s["scales"], c["K"], s["table"], s["starts"], s["rows"], first=s["first"], out=s["out"])
    if c["op"] == "attention":
        return dsnq.paged_latent_attention_fp8(s["q"], s["cache"], s["scales"], s["table"], s["lens"], c["DV"], s["scale"],
                                               out=s["out"], lse=s["lse"])
    return dsnq.shared_prefix_latent_attention_fp8(s["q"], s["cache"], s["scales"], s["prefix_table"], s["prefix_len"], s["table"],
                                                   s["lens"], c["DV"], s["scale"], out=s["out"], lse=s["lse"])


def run(state):
    return _own(state) if own else _PLAIN[state["c"]["op"]](state)


# ----------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, K, P = s["c"], s["c"]["K"], s["c"]["P"]
    if c["op"] == "write":
        kv = s["kv"].double()
        if c["norm"]:
            kv = kv / kv.square().mean(-1, keepdim=True).add(EPS).sqrt() * s["gamma"].double()
        x = kv.clone() if s["pe"] is None else torch.cat([kv, s["pe"].double()], -1)
        z = torch.polar(torch.ones(c["M"], 32, dtype=torch.float64, device=DEV), s["positions"][:, None].double() * s["inv_freq"][None])
        v = x[:, s["off"]:]
        if c["layout"] == "half":
            w = torch.complex(v[:, :32].contiguous(), v[:, 32:].contiguous()) * z
            v = torch.cat([w.real, w.imag], -1)
        else:
            v = torch.view_as_real(torch.view_as_complex(v.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        x[:, s["off"]:] = v
        scale = torch.clamp(x[:, :K].abs().max(-1).values / TOP, min=LEAST)
        x = x / scale[:, None]
        codes, pe, scales = (t.double() for t in _views(s))
        keep = s["slots"] >= 0
        for whole, new in ((codes, x[:, :K]), (pe, x[:, K:]), (scales[..., None], scale[:, None])):
            if new.shape[1]:
                whole.view(-1, new.shape[1])[s["slots"][keep]] = new[keep]
        return codes, pe, scales

    def held(pages, first, end):
        """Tokens [first, end) of the pages, in 64 bits."""
        rows = s["cache"][pages.long()].reshape(-1, K + 2 * P)[first:end]
        scale = s["scales"][pages.long()].reshape(-1)[first:end].double()
        return torch.cat([rows[:, :K].view(torch.float8_e4m3fn).double(), rows[:, K:].contiguous().view(torch.bfloat16).double()], -1) * scale[:, None]

    lens, page = _lens(c), c["page"]
    if c["op"] == "read":
        out, at = s["out"].double(), 0
        for b, (n, f) in enumerate(zip(lens, _firsts(c))):
            out[at:at + n - f] = held(s["table"][b, :-(-n // page)], f, n)
            at += n - f
        return out
    out = torch.zeros(c["B"], c["H"], c["DV"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    front = held(s["prefix_table"], 0, c["prefix"]) if c["op"] == "shared" else None
    for b, n in enumerate(lens):
        k = held(s["table"][b, :-(-n // page)], 0, n)
        if front is not None:
            k = torch.cat([front, k])
        if not k.shape[0]:
            continue
        z = (s["q"][b].double() @ k.T) * s["scale"]
        lse[b] = torch.logsumexp(z, -1)
        out[b] = torch.exp(z - lse[b][:, None]) @ k[:, :c["DV"]]
    return out, lse
