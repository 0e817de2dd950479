"""The operators of a decode step around the latent pre-projection, each in its
plain form and as the library's call, over the sizes they are used at.

  extend_block_tables     block tables, positions and slots from request lengths
  head_rmsnorm_rope       per-head RMSNorm and rotary positions in one pass
  latent_cache_write      normalized and rotated latent rows into the paged cache
  paged_latent_attention  one new token per request over the paged latent cache

run(state) makes one pass: elementary torch operations in fp32 (rotary angles
in fp64) where `own` is false, the library's entry point where it is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # A decode step of a serving batch: every request grows by one token.
        {"name": "extend decode 48", "op": "extend", "B": 48, "prompts": 0, "chunk": 0, "page": 64, "maxlen": 16384, "shape": 1},
        # Mixed batch: many decoding requests and prompts that arrive in chunks, padded rows at the end.
        {"name": "extend mixed 1000", "op": "extend", "B": 1000, "prompts": 40, "chunk": 1021, "page": 16, "maxlen": 32768, "shape": 2},
        # One decode token: rotation of the last 64 of each attention head's 192 columns (128 heads).
        {"name": "rope decode 1", "op": "rope", "M": 1, "H": 128, "D": 192, "R": 64, "off": 128, "norm": 0, "gamma": 0,
         "layout": "interleaved", "maxpos": 4096, "factor": 1.0, "wide": 0},
        # Indexer heads of a small odd batch, weighted norm, half-split pairs, rows inside a wider buffer.
        {"name": "rope indexer 77", "op": "rope", "M": 77, "H": 32, "D": 128, "R": 64, "off": 64, "norm": 1, "gamma": 1,
         "layout": "half", "maxpos": 131072, "factor": 1.0, "wide": 1},
        # Prompt tokens far into a long context, scaled frequencies, whole-head norm of 48 heads of 512.
        {"name": "rope prompt 4096", "op": "rope", "M": 4096, "H": 48, "D": 512, "R": 64, "off": 448, "norm": 1, "gamma": 0,
         "layout": "interleaved", "maxpos": 1000000, "factor": 16.0, "wide": 0},
        # Decode batch: the normalized latent of the pre-projection and the 64 position columns of its row.
        {"name": "write decode 32", "op": "write", "M": 32, "K": 512, "P": 64, "R": 64, "norm": 0, "layout": "interleaved",
         "page": 64, "maxpos": 16384, "factor": 1.0, "pad": 3},
        # Prompt: raw latents, normalized on the way into the cache, a few padded rows.
        {"name": "write prompt 8191", "op": "write", "M": 8191, "K": 512, "P": 64, "R": 64, "norm": 1, "layout": "interleaved",
         "page": 64, "maxpos": 131072, "factor": 4.0, "pad": 17},
        # One request of a chat, all 128 heads: the latency of a single decode.
        {"name": "attention 1 x 701", "op": "attention", "B": 1, "H": 128, "DK": 576, "DV": 512, "page": 64, "maxlen": 701,
         "even": 1, "empty": 0, "shape": 3},
        # Two long documents with a sixteenth of the heads on this GPU, small pages: split over the length.
        {"name": "attention 2 x 131071", "op": "attention", "B": 2, "H": 16, "DK": 576, "DV": 512, "page": 32, "maxlen": 131071,
         "even": 1, "empty": 0, "shape": 4},
        # Serving batch of mixed lengths, all heads, a padded (empty) row in it.
        {"name": "attention 40 mixed", "op": "attention", "B": 40, "H": 128, "DK": 576, "DV": 512, "page": 64, "maxlen": 4096,
         "even": 0, "empty": 2, "shape": 5},
        # Large even batch, 48 heads as wide as the latent, keys and values the same 512 columns: the most bytes.
        {"name": "attention 128 x 8000", "op": "attention", "B": 128, "H": 48, "DK": 512, "DV": 512, "page": 16, "maxlen": 8000,
         "even": 1, "empty": 0, "shape": 6},
        # Large batch, all heads, lengths from a few tokens to a long context: uneven work for the GPU.
        {"name": "attention 96 mixed", "op": "attention", "B": 96, "H": 128, "DK": 576, "DV": 512, "page": 64, "maxlen": 32768,
         "even": 0, "empty": 1, "shape": 7},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "rope", "write", "attention", "attention"])
    if op == "extend":
        B = _log(rng, 1, 1000)
        return {"op": op, "B": B, "prompts": rng.choice([0, min(B, 1 + B // 25)]), "chunk": _log(rng, 2, 1000),
                "page": rng.choice([8, 16, 32, 64, 128]), "maxlen": _log(rng, 200, 32768), "shape": rng.randrange(1 << 20)}
    if op == "rope":
        H, D = rng.choice([(128, 192), (32, 128), (48, 512), (16, 64), (3, 256), (16, 192), (1, 576)])
        R = rng.choice([32, 64])
        norm = rng.randrange(2)
        return {"op": op, "M": _log(rng, 1, 4096), "H": H, "D": D, "R": R, "off": rng.choice([0, D - R]), "norm": norm,
                "gamma": norm and rng.randrange(2), "layout": rng.choice(["interleaved", "half"]),
                "maxpos": _log(rng, 100, 2000000), "factor": rng.choice([1.0, 4.0, 16.0]), "wide": rng.randrange(2)}
    if op == "write":
        K, P = rng.choice([(512, 64), (512, 64), (512, 0), (256, 64)])
        M = _log(rng, 1, 8000)
        return {"op": op, "M": M, "K": K, "P": P, "R": 64, "norm": rng.randrange(2),
                "layout": rng.choice(["interleaved", "half"]), "page": rng.choice([16, 32, 64, 128]),
                "maxpos": _log(rng, 100, 2000000), "factor": rng.choice([1.0, 4.0, 16.0]), "pad": rng.randrange(0, min(M, 9))}
    DK, DV = rng.choice([(576, 512), (576, 512), (512, 512), (320, 256)])
    B = _log(rng, 1, 96)
    return {"op": op, "B": B, "H": rng.choice([1, 8, 16, 24, 48, 64, 100, 128]), "DK": DK, "DV": DV,
            "page": rng.choice([8, 16, 32, 48, 64, 128, 256]), "maxlen": _log(rng, 1, min(100000, 400000 // B)),
            "even": rng.randrange(2), "empty": rng.randrange(0, 1 + B // 8), "shape": rng.randrange(1 << 20)}


def _lens(c):
    """Request lengths of an attention case."""
    r = random.Random(c["shape"])
    lens = [c["maxlen"] if c["even"] else _log(r, 1, c["maxlen"]) for _ in range(c["B"])]
    for i in range(c["empty"]):
        lens[(7 * i + 3) % c["B"]] = 0
    return lens


def _extend_lens(c):
    """(lengths so far, new tokens) of an extend case."""
    r = random.Random(c["shape"])
    old = [_log(r, 1, c["maxlen"]) for _ in range(c["B"])]
    new = [1] * c["B"]
    for b in r.sample(range(c["B"]), c["prompts"]):
        new[b] = r.randrange(2, c["chunk"] + 1)
        old[b] = r.choice([0, old[b]])
    return old, new


def _extend_rows(c):
    return sum(_extend_lens(c)[1]) + c["B"] % 8          # padded rows at the end


def work(case):
    c = case
    if c["op"] == "extend":
        old, new = _extend_lens(c)
        pages = sum(-(-(o + n) // c["page"]) - -(-o // c["page"]) for o, n in zip(old, new))
        partial = sum(1 for o in old if o % c["page"])
        # lengths and counts in, lengths and row starts out, page ids in and into the table, positions and slots out
        return {"bytes": 16 * c["B"] + 8 * pages + 4 * partial + 16 * _extend_rows(c), "flops": 0}
    if c["op"] == "rope":
        n = c["M"] * c["H"] * c["D"]
        return {"bytes": 4 * n + 8 * c["M"] + 4 * c["R"] + 2 * c["D"] * c["gamma"],
                "flops": (4 * n if c["norm"] else 0) + 3 * c["M"] * c["H"] * c["R"]}
    if c["op"] == "write":
        live, W = c["M"] - c["pad"], c["K"] + c["P"]
        return {"bytes": 4 * live * W + 8 * c["M"] + 8 * live + 4 * c["R"] + 2 * c["K"] * c["norm"],
                "flops": live * (4 * c["K"] * c["norm"] + 3 * c["R"])}
    total = sum(_lens(c))
    pages = sum(-(-n // c["page"]) for n in _lens(c))
    return {"bytes": 2 * total * c["DK"] + 4 * pages + 2 * c["B"] * c["H"] * (c["DK"] + c["DV"]) + 4 * c["B"] * (c["H"] + 1),
            "flops": 2 * total * c["H"] * (c["DK"] + c["DV"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _ints(n, dtype=torch.int32):
    return torch.empty(n, dtype=dtype, device=DEV)


def _inv_freq(R, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Rotary frequencies [R/2] in fp64 and the factor of cos and sin.  With
    factor > 1 the slow ones are divided by it and the fast ones kept, with a
    linear ramp between (a context `factor` times the original)."""
    i = torch.arange(0, R, 2, dtype=torch.float64, device=DEV)
    f = base ** (-i / R)
    if factor <= 1.0:
        return f, 1.0
    dim = [R * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
    low, high = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), R - 1)
    ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    """Inputs, and the output buffers that a decode loop keeps from step to step."""
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    if c["op"] == "extend":
        old, new = _extend_lens(c)
        page = c["page"]
        held = [-(-o // page) for o in old]
        width = max(-(-(o + n) // page) for o, n in zip(old, new)) + 1
        need = sum(-(-(o + n) // page) for o, n in zip(old, new)) - sum(held)
        pool = torch.randperm(sum(held) + need + 32, generator=g, device=DEV).to(torch.int32)
        h = torch.tensor(held, device=DEV)
        col = torch.arange(width, device=DEV)
        mine = col[None] < h[:, None]
        table = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
        table[mine] = pool[:sum(held)]
        s.update(seq_lens=torch.tensor(old, dtype=torch.int32, device=DEV), new_tokens=torch.tensor(new, dtype=torch.int32, device=DEV),
                 table=table, free=pool[sum(held):].contiguous(), rows=_extend_rows(c),
                 out=(_ints(c["B"]), _ints(c["B"] + 1), _ints(_extend_rows(c), torch.int64), _ints(_extend_rows(c), torch.int64), _ints(2)))
        return s
    if c["op"] == "attention":
        lens = _lens(c)
        page = c["page"]
        held = [-(-n // page) for n in lens]
        width = max(max(held), 1) + 1
        pool = torch.randperm(sum(held) + 4, generator=g, device=DEV).to(torch.int32)
        mine = torch.arange(width, device=DEV)[None] < torch.tensor(held, device=DEV)[:, None]
        table = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
        table[mine] = pool[:sum(held)]
        gamma = torch.rand(c["DK"], generator=g, device=DEV) + 0.5
        cache = _randn(g, sum(held) + 4, page, c["DK"])
        cache.mul_(gamma.to(torch.bfloat16))
        s.update(q=_randn(g, c["B"], c["H"], c["DK"]), cache=cache, table=table,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scale=(c["DK"] / 3.0) ** -0.5,
                 out=torch.empty(c["B"], c["H"], c["DV"], dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(c["B"], c["H"], dtype=torch.float32, device=DEV))
        return s
    f, m = _inv_freq(c["R"], c["factor"])
    first = torch.randint(0, c["maxpos"], (1,), generator=g, device=DEV)
    spread = torch.randint(0, c["maxpos"], (c["M"],), generator=g, device=DEV)
    run = (first + torch.arange(c["M"], device=DEV)) % c["maxpos"]
    s.update(inv_freq=f, rope_scale=m, positions=spread if c["M"] < 512 else run)   # decode batches and prompts
    if c["op"] == "rope":
        H, D = c["H"], c["D"]
        buf = _randn(g, c["M"], H * D + (64 if c["wide"] else 0))
        s.update(x=buf[:, :H * D].view(c["M"], H, D), out=torch.empty(c["M"], H, D, dtype=torch.bfloat16, device=DEV),
                 gamma=(torch.rand(D, generator=g, device=DEV) + 0.5).to(torch.bfloat16) if c["gamma"] else None)
        return s
    K, P, M, page = c["K"], c["P"], c["M"], c["page"]
    row = _randn(g, M, 1536 + K + P)                     # the fused projection's row: q latent, kv latent, position columns
    pages = -(-M // page) + 4
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:M]
    if c["pad"]:
        slots[M - c["pad"]:] = -1
    s.update(kv=row[:, 1536:1536 + K], pe=row[:, 1536 + K:] if P else None, slots=slots,
             gamma=(torch.rand(K, generator=g, device=DEV) + 0.5).to(torch.bfloat16) if c["norm"] else None,
             cache=_randn(g, pages, page, K + P), off=K + P - c["R"])
    return s


# ------------------------------------------------------------- plain forms

def _rotate(v, cos, sin, layout):
    """v [..., R] rotated by the angles of cos, sin [..., R/2]."""
    if layout == "half":
        a, b = v.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = v[..., 0::2], v[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    return (angle.cos() * s["rope_scale"]).float(), (angle.sin() * s["rope_scale"]).float()


def _rms(x, gamma):
    x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS))
    return x if gamma is None else x * gamma.float()


def _plain_extend(s):
    page, table, rows = s["c"]["page"], s["table"], s["rows"]
    cap = table.shape[1] * page
    old = s["seq_lens"].long().clamp(0, cap)
    want = s["new_tokens"].long().clamp(min=0)
    end = want.cumsum(0)
    start = end - want
    fit = torch.minimum(torch.minimum(want, (rows - start).clamp(min=0)), cap - old)
    held = (old + page - 1) // page
    need = (old + fit + page - 1) // page - held
    first = need.cumsum(0) - need
    F = s["free"].numel()
    got = torch.minimum(need, (F - first).clamp(min=0))
    new_lens = torch.minimum(old + fit, (held + got) * page)
    col = torch.arange(table.shape[1], device=DEV)[None]
    k = col - held[:, None]
    fresh = (k >= 0) & (k < got[:, None])
    table.copy_(torch.where(fresh, s["free"][(first[:, None] + k).clamp(0, F - 1)], table))
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(end, r, right=True)
    live = b < old.numel()
    b = b.clamp(max=old.numel() - 1)
    pos = torch.where(live, old[b] + r - start[b], 0)
    entry = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (pos < new_lens[b]) & (entry >= 0), entry * page + pos % page, -1)
    row_starts = torch.cat([start, end[-1:]]).clamp(max=rows).int()
    counts = torch.stack([got.sum(), need.sum()]).int()
    return new_lens.int(), row_starts, pos, slots, counts, table


def _plain_rope(s):
    c = s["c"]
    x = s["x"].float()
    if c["norm"]:
        x = _rms(x, s["gamma"])
    cos, sin = _cos_sin(s)
    lo, hi = c["off"], c["off"] + c["R"]
    y = _rotate(x[..., lo:hi], cos[:, None], sin[:, None], c["layout"])
    return torch.cat([x[..., :lo], y, x[..., hi:]], -1).bfloat16()


def _plain_write(s):
    c, cache = s["c"], s["cache"]
    x = s["kv"].float()
    if c["norm"]:
        x = _rms(x, s["gamma"])
    if s["pe"] is not None:
        x = torch.cat([x, s["pe"].float()], -1)
    cos, sin = _cos_sin(s)
    row = torch.cat([x[:, :s["off"]], _rotate(x[:, s["off"]:], cos, sin, c["layout"])], -1).bfloat16()
    flat = cache.view(-1, cache.shape[-1])
    at = s["slots"].clamp(min=0)
    # Rows without a slot land on row 0 of a copy that is one row longer.
    longer = torch.cat([flat, flat[:1]])
    longer[torch.where(s["slots"] >= 0, at, flat.shape[0])] = row
    flat.copy_(longer[:-1])
    return cache


def _plain_attention(s):
    c, cache, lens, table = s["c"], s["cache"], s["lens"], s["table"]
    page = c["page"]
    n = table.shape[1] * page
    at = torch.arange(n, device=DEV)
    valid = at[None] < lens[:, None]
    rows = table.long().clamp(min=0)[:, at // page] * page + at % page
    k = cache.view(-1, c["DK"])[rows].float()
    k = torch.where(valid[..., None], k, 0.0)
    score = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    score = torch.where(valid[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, k[..., :c["DV"]]) / torch.where(total > 0, total, 1.0)
    return out.bfloat16(), (top + torch.log(total))[..., 0]


_PLAIN = {"extend": _plain_extend, "rope": _plain_rope, "write": _plain_write, "attention": _plain_attention}


# ------------------------------------------------------- the library's calls

def _own(s):
    import gemm_dsnq_dual_gb300 as dsnq
    c = s["c"]
    if c["op"] == "extend":
        return *dsnq.extend_block_tables(s["seq_lens"], s["new_tokens"], s["free"], s["table"], c["page"], s["rows"], out=s["out"]), s["table"]
    if c["op"] == "rope":
        return dsnq.head_rmsnorm_rope(s["x"], s["positions"], s["inv_freq"], gamma=s["gamma"], eps=EPS, normalize=bool(c["norm"]),
                                      rope_offset=c["off"], layout=c["layout"], rope_scale=s["rope_scale"], out=s["out"])
    if c["op"] == "write":
        return dsnq.latent_cache_write(s["kv"], s["pe"], s["positions"], s["slots"], s["inv_freq"], s["cache"], gamma=s["gamma"],
                                       eps=EPS, normalize=bool(c["norm"]), rope_offset=s["off"], layout=c["layout"],
                                       rope_scale=s["rope_scale"])
    return dsnq.paged_latent_attention(s["q"], s["cache"], s["table"], s["lens"], c["DV"], s["scale"], out=s["out"], lse=s["lse"])


def run(state):
    return _own(state) if own else _PLAIN[state["c"]["op"]](state)


# ----------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "extend":
        return None                                      # whole numbers only
    if c["op"] == "attention":
        out = torch.zeros(c["B"], c["H"], c["DV"], dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(c)):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // c["page"])].long()
            k = s["cache"][pages].reshape(-1, c["DK"])[:n].double()
            z = (s["q"][b].double() @ k.T) * s["scale"]
            lse[b] = torch.logsumexp(z, -1)
            out[b] = torch.exp(z - lse[b][:, None]) @ k[:, :c["DV"]]
        return out, lse
    z = torch.polar(torch.full((c["M"], c["R"] // 2), float(s["rope_scale"]), dtype=torch.float64, device=DEV),
                    s["positions"][:, None].double() * s["inv_freq"][None])

    def turn(v, z):
        if c["layout"] == "interleaved":
            return torch.view_as_real(torch.view_as_complex(v.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        w = torch.complex(v[..., :c["R"] // 2].contiguous(), v[..., c["R"] // 2:].contiguous()) * z
        return torch.cat([w.real, w.imag], -1)

    if c["op"] == "rope":
        x = s["x"].double().clone()
        if c["norm"]:
            x = x / x.square().mean(-1, keepdim=True).add(EPS).sqrt()
            if s["gamma"] is not None:
                x = x * s["gamma"].double()
        x[..., c["off"]:c["off"] + c["R"]] = turn(x[..., c["off"]:c["off"] + c["R"]], z[:, None])
        return x
    kv = s["kv"].double()
    if c["norm"]:
        kv = kv / kv.square().mean(-1, keepdim=True).add(EPS).sqrt() * s["gamma"].double()
    x = kv if s["pe"] is None else torch.cat([kv, s["pe"].double()], -1)
    x = x.clone()
    x[:, s["off"]:] = turn(x[:, s["off"]:], z)
    cache = s["cache"].double()
    keep = s["slots"] >= 0
    cache.view(-1, c["K"] + c["P"])[s["slots"][keep]] = x[keep]
    return cache
