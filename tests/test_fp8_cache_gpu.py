"""The latent cache in 8 bits on the GPU against plain implementations in 64
bits: its write, its read, the paged attention over it, the attention behind a
prefix that all requests share, and a run of them.

Tolerances.  Write: before its rounding a row's fp32 arithmetic is off by at
most 2^-14 of |a| + |b| of the rotated pairs (norm 2^-15, angles and products
2^-21), the rounding by half a step: 2^-4 of a code's value or 2^-10 (below the
normal numbers), 2^-8 of a position column.  Read: exact (one fp32 product, one
rounding).  Attention: the weight p s of a token becomes two e4m3 numbers, off
by at most 2^-8 of itself or 2^-21 of the largest weight among the 32 tokens it
is multiplied with; the output is divided by the sum of the p that they stand
for, so these errors act on the distance of a value from the output; a score is
off by at most dz = ((DK / 32 + 8) 2^-23) of the largest sum of |q k| * scale
(an fp32 addition per 32-wide step of the tensor core, whose additions
truncate, and fp32 scalings) and 2^-23 of the head's largest |q| times the sum
of |k| (what the split of q leaves), which moves every probability by 2 dz;
sums and exponentials add 2^-18.  The output is rounded to bf16: 2^-8."""

import math
import sys

import numpy as np
import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq

pytestmark = pytest.mark.gpu
OK, TIMEOUT, BOUNDS = 0, 5, 6
DEV = "cuda"
I32, I64, BF, F32, F64, U8, E4 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


def make_cache(g, pages, page, K, P, spread=0.0, ld_row=None):
    """(cache, scales): random codes and position columns; scales 2^N(-8, spread)."""
    W = K + 2 * P
    cache = torch.empty(pages, page, ld_row or W, dtype=U8, device=DEV)[..., :W]
    cache[..., :K] = (torch.randn(pages, page, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4).view(U8)
    if P:
        cache[..., K:] = (torch.randn(pages, page, P, generator=g, device=DEV) * 100).to(BF).view(U8)
    return cache, torch.exp2(-8 + spread * torch.randn(pages, page, generator=g, device=DEV))


def values(cache, scales, K):
    """The rows that a cache stands for, in 64 bits: [pages * page, K + P]."""
    c = cache.contiguous()
    parts = [c[..., :K].view(E4).double()] + ([c[..., K:].contiguous().view(BF).double()] if c.shape[-1] > K else [])
    return (torch.cat(parts, -1) * scales.double()[..., None]).flatten(0, 1)


def slots_of(table, page, first, end):
    at = torch.arange(first, end, device=DEV)
    return table.long()[at // page] * page + at % page


# ---------------------------------------------------------------------- write

def rotated(x, positions, freq, off, layout):
    """x [M, W] fp64 with its pairs rotated, and |a| + |b| of each column's pair (0 elsewhere)."""
    R = 2 * freq.numel()
    v = x[:, off:off + R]
    ang = positions.double()[:, None] * freq                   # positions are small here
    c, s = ang.cos(), ang.sin()
    a, b = (v[:, 0::2], v[:, 1::2]) if layout == "interleaved" else (v[:, :R // 2], v[:, R // 2:])
    lo, hi, both = a * c - b * s, b * c + a * s, a.abs() + b.abs()
    out, pair = x.clone(), x.abs()
    for t, (p, q) in ((out, (lo, hi)), (pair, (both, both))):
        t[:, off:off + R] = torch.stack([p, q], -1).flatten(1) if layout == "interleaved" else torch.cat([p, q], -1)
    return out, pair


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,K,P,R,off,page,norm", [
    (1, 512, 64, 64, 512, 64, True), (77, 512, 64, 64, 512, 16, False), (300, 512, 0, 64, 448, 48, True), (33, 256, 64, 32, 0, 8, True),
    (130, 16, 8, 16, 8, 13, True), (5, 1024, 0, 256, 256, 1, True), (64, 960, 64, 64, 928, 64, False), (9, 512, 64, 0, 0, 64, False)])
def test_write(M, K, P, R, off, page, norm, layout):
    g = gen(M + K + page)
    row = randn(g, M, K + P + 24)
    kv, pe = row[:, :K], row[:, K:K + P] if P else None
    gamma = (torch.rand(K, generator=g, device=DEV) + 0.5).to(BF) if norm else None
    positions = torch.randint(0, 5000, (M,), generator=g, device=DEV)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=F64, device=DEV) / max(R, 1))
    pages = -(-M // page) + 3
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:M]
    if M > 4:
        slots[[1, M - 1]] = -1
    buf = torch.randint(0, 256, (pages, page, K + 2 * P + 32), generator=g, device=DEV, dtype=I32).to(U8)
    cache, scales = buf[..., :K + 2 * P], torch.rand(pages, page + 4, generator=g, device=DEV)[:, :page]
    before, before_s = buf.clone(), scales.clone()
    got = dsnq.latent_cache_write_fp8(kv, pe, positions, slots, freq, cache, scales, gamma=gamma, normalize=norm,
                                      rope_offset=off, layout=layout)
    assert got[0] is cache and got[1] is scales and dsnq.debug_status() == OK
    x = kv.double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gamma.double()
    if P:
        x = torch.cat([x, pe.double()], -1)
    x, pair = rotated(x, positions, freq, off, layout) if R else (x, x.abs())
    keep = slots >= 0
    at, x, pair = slots[keep], x[keep], pair[keep]
    s = scales.reshape(-1)[at].double()
    noise = 2.0 ** -14 * pair
    top = x[:, :K].abs().amax(-1)
    assert ((s - top / 448).abs() <= (noise[:, :K].amax(-1) + 2.0 ** -22 * top) / 448).all()
    flat = cache.reshape(-1, K + 2 * P)[at]
    codes = flat[:, :K].contiguous().view(E4).double() * s[:, None]
    bound = 2.0 ** -4 * x[:, :K].abs() + 2.0 ** -10 * s[:, None] + noise[:, :K] * 1.1
    assert ((codes - x[:, :K]).abs() <= bound).all()
    if P:
        pos = flat[:, K:].contiguous().view(BF).double() * s[:, None]
        assert ((pos - x[:, K:]).abs() <= 2.0 ** -8 * x[:, K:].abs() + noise[:, K:] * 1.1 + 1e-30).all()
    # Nothing else has changed: other rows, and what lies between rows and pages.
    untouched = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    untouched[at] = False
    assert torch.equal(buf.view(-1, buf.shape[-1])[untouched], before.view(-1, buf.shape[-1])[untouched])
    assert torch.equal(buf[..., K + 2 * P:], before[..., K + 2 * P:])
    assert torch.equal(scales.reshape(-1)[untouched], before_s.reshape(-1)[untouched])


def test_write_codes_are_those_of_the_division():
    """Without norm and rotation a row's scale and codes are exact: IEEE
    quotients, rounded to nearest, ties to even."""
    g = gen(3)
    kv = (randn(g, 4000, 512).float() * torch.exp2(torch.randint(-40, 40, (4000, 1), generator=g, device=DEV).float())).to(BF)
    cache, scales = torch.zeros(63, 64, 512, dtype=U8, device=DEV), torch.zeros(63, 64, device=DEV)
    dsnq.latent_cache_write_fp8(kv, None, torch.zeros(4000, dtype=I64, device=DEV), torch.arange(4000, device=DEV),
                                torch.empty(0, dtype=F64, device=DEV), cache, scales)
    # (In 64 bits and rounded to 32: the fp32 quotient.  torch divides fp32 by a number by multiplying.)
    x = kv.double()
    s = (x.abs().amax(-1) / 448.0).clamp(min=2.0 ** -60).float()
    assert torch.equal(scales.view(-1)[:4000], s)
    assert torch.equal(cache.view(-1, 512)[:4000], (x / s.double()[:, None]).float().to(E4).view(U8))


def test_write_position_columns_are_those_of_the_division():
    g = gen(21)
    M, K, P = 5000, 16, 64
    kv = randn(g, M, K) * torch.exp(torch.randn(M, 1, generator=g, device=DEV) * 8).to(BF)
    pe = randn(g, M, P) * torch.exp(torch.randn(M, P, generator=g, device=DEV) * 8).to(BF)
    cache, scales = torch.zeros(M // 8, 8, K + 2 * P, dtype=U8, device=DEV), torch.zeros(M // 8, 8, device=DEV)
    at = torch.randperm(M, generator=g, device=DEV)
    dsnq.latent_cache_write_fp8(kv, pe, torch.zeros(M, dtype=I64, device=DEV), at, torch.empty(0, dtype=F64, device=DEV), cache, scales)
    s = scales.flatten()[at]
    want = (pe.double() / s.double()[:, None]).float().to(BF)  # the 64-bit quotient rounds to 32 bits as the exact one does
    got = cache.view(-1, K + 2 * P)[at, K:].contiguous().view(BF)
    assert torch.equal(got, want) and dsnq.debug_status() == OK


def test_write_zero_tiny_and_non_finite_rows():
    K, P = 256, 64
    kv = torch.zeros(7, K, dtype=BF, device=DEV)
    pe = torch.full((7, P), 3.0, dtype=BF, device=DEV)
    kv[1, 5] = 1e-30                                           # below the least scale: codes 0
    kv[2, 7], kv[3, 9], kv[4, 11] = math.nan, math.inf, -math.inf
    kv[5, 3], pe[5, 2] = 1.0, math.nan                         # NaN among the position columns stays there
    kv[6, 0] = 3.0e38
    cache, scales = torch.zeros(1, 8, K + 2 * P, dtype=U8, device=DEV), torch.zeros(1, 8, device=DEV)
    at = torch.arange(7, device=DEV)
    dsnq.latent_cache_write_fp8(kv, pe, torch.zeros(7, dtype=I64, device=DEV), at, torch.empty(0, dtype=F64, device=DEV), cache, scales)
    out = dsnq.latent_cache_read_fp8(cache, scales, K, ints([[0]]), ints([0, 7]), 7)
    assert (out[:2, :K] == 0).all() and (out[:2, K:] == 3).all() and (scales[0, :2] == 2.0 ** -60).all()
    assert out[2:5].isnan().all()
    assert out[5].isnan().sum() == 1 and out[5, K + 2].isnan() and out[5, 3] == 1
    assert out[6, 0] == kv[6, 0] and (out[6, K:].float() - 3).abs().max() <= 3 * 2.0 ** -7
    assert dsnq.debug_status() == OK


def test_write_reports_a_slot_past_the_cache():
    cache, scales = torch.zeros(2, 8, 256, dtype=U8, device=DEV), torch.zeros(2, 8, device=DEV)
    kv = torch.ones(3, 256, dtype=BF, device=DEV)
    dsnq.latent_cache_write_fp8(kv, None, torch.zeros(3, dtype=I64, device=DEV), torch.tensor([3, 16, -9], device=DEV),
                                torch.empty(0, dtype=F64, device=DEV), cache, scales)
    assert dsnq.debug_status() == BOUNDS and dsnq.debug_status() == OK
    assert (scales != 0).sum() == 1 and (cache != 0).any(-1).sum() == 1


# ----------------------------------------------------------------------- read

@pytest.mark.parametrize("K,P,page,lens,first", [
    (512, 64, 64, [1, 0, 130, 64, 7], None), (512, 64, 16, [700, 1, 33], [699, 0, 5]), (256, 64, 8, [0, 0, 9], None),
    (512, 0, 48, [1000], [17]), (16, 8, 13, [40, 3], [1, 1]), (1024, 0, 64, [5, 70], None), (960, 64, 1, [3, 6], [2, 0])])
def test_read(K, P, page, lens, first):
    g = gen(K + page)
    held = [-(-n // page) for n in lens]
    cache, scales = make_cache(g, sum(held) + 2, page, K, P, spread=3, ld_row=K + 2 * P + 48)
    wide = torch.full((len(lens), max(held) + 5), -7, dtype=I32, device=DEV)
    table = wide[:, 2:2 + max(held)]
    ids = torch.randperm(sum(held) + 2, generator=g, device=DEV).to(I32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    f = first or [0] * len(lens)
    counts = [n - x for n, x in zip(lens, f)]
    starts = np.concatenate([[0], np.cumsum(counts)])
    rows = int(starts[-1]) + 5
    buf = randn(g, rows, K + P + 8)
    want = buf.clone()
    v = values(cache, scales, K).float().to(BF)                # one product exact in 64 bits, in 32 bits rounded as here
    codes = cache.contiguous()[..., :K].view(E4).float() * scales[..., None]
    v = codes.to(BF) if not P else torch.cat([codes, cache.contiguous()[..., K:].contiguous().view(BF).float() * scales[..., None]], -1).to(BF)
    v = v.flatten(0, 1)
    for b in range(len(lens)):
        if counts[b]:
            want[starts[b]:starts[b + 1], :K + P] = v[slots_of(table[b], page, f[b], lens[b])]
    out = dsnq.latent_cache_read_fp8(cache, scales, K, table, ints(starts.tolist()), rows, first=None if first is None else ints(first),
                                     out=buf[:, :K + P])
    assert torch.equal(buf, want) and dsnq.debug_status() == OK and out.data_ptr() == buf.data_ptr()
    fresh = dsnq.latent_cache_read_fp8(cache, scales, K, table, ints(starts.tolist()), rows, first=None if first is None else ints(first))
    assert torch.equal(fresh[:starts[-1]], want[:starts[-1], :K + P])


def test_read_outside_the_table_and_bad_pages():
    """Zeros, and a report; neighbours are what they are."""
    cache, scales = make_cache(gen(1), 4, 8, 256, 0)
    table = ints([[0, 9], [-1, 2]])
    out = dsnq.latent_cache_read_fp8(cache, scales, 256, table, ints([0, 20, 36]), 36)
    assert dsnq.debug_status() == BOUNDS
    v = (cache.view(E4).float() * scales[..., None]).to(BF)
    assert torch.equal(out[:8], v[0]) and (out[8:20] == 0).all() and (out[20:28] == 0).all() and torch.equal(out[28:36], v[2])
    out = dsnq.latent_cache_read_fp8(cache, scales, 256, ints([[1, 3]]), ints([2, 5]), 7, first=ints([-1]), out=torch.ones(7, 256, dtype=BF, device=DEV))
    assert dsnq.debug_status() == BOUNDS
    assert (out[:2] == 1).all() and (out[2] == 0).all() and torch.equal(out[3:5], v[1, :2]) and (out[5:] == 1).all()


def test_read_largest_batch_and_empty_calls():
    B = 8192
    cache, scales = make_cache(gen(2), 64, 8, 16, 0)
    lens = (torch.arange(B, device=DEV) % 3).to(I32)
    table = (torch.arange(B, device=DEV) % 64).to(I32)[:, None]
    starts = torch.cat([torch.zeros(1, dtype=I32, device=DEV), lens.cumsum(0).to(I32)])
    rows = int(starts[-1])
    out = dsnq.latent_cache_read_fp8(cache, scales, 16, table, starts, rows)
    v = (cache.view(E4).float() * scales[..., None]).to(BF)
    b = torch.repeat_interleave(torch.arange(B, device=DEV), lens.long())
    assert torch.equal(out, v[b % 64, torch.arange(rows, device=DEV) - starts.long()[b]])
    assert dsnq.latent_cache_read_fp8(cache, scales, 16, table, starts, 0).shape == (0, 16)
    one = torch.full((3, 16), 2.0, dtype=BF, device=DEV)
    dsnq.latent_cache_read_fp8(cache, scales, 16, torch.empty(0, 4, dtype=I32, device=DEV), ints([0]), 3, out=one)
    assert (one == 2).all() and dsnq.debug_status() == OK


# ------------------------------------------------------------------ attention

def reference(q, rows, codes_abs, weights_scale, scale, v_dim):
    """One request in 64 bits: out [H, DV], lse [H] and their bounds.  rows
    [n, DK] values of its tokens; codes_abs [n, DV] |codes|, weights_scale [n]
    the scales (for the bound of small weights)."""
    H, DK = q.shape
    if rows.shape[0] == 0:
        z = torch.zeros(H, v_dim, dtype=F64, device=DEV)
        return z, torch.full((H,), -math.inf, dtype=F64, device=DEV), z, torch.zeros(H, dtype=F64, device=DEV)
    z = scale * q @ rows.T
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    v = rows[:, :v_dim]
    out = p @ v
    reach = (scale * q.abs() @ rows.abs().T).amax(-1)
    dz = (DK / 32 + 8) * 2.0 ** -23 * reach + 2.0 ** -23 * scale * q.abs().amax(-1) * rows.abs().sum(-1).max()
    small = torch.zeros(H, v_dim, dtype=F64, device=DEV)
    w = p * weights_scale
    for at in range(0, rows.shape[0], 32):
        small += w[:, at:at + 32].amax(-1, keepdim=True) * codes_abs[at:at + 32].sum(0)
    far = p @ v.abs() + out.abs()
    bound = (2.0 ** -8 + 2 * dz[:, None] + 2.0 ** -17) * far + 2.0 ** -21 * small + 2.0 ** -8 * out.abs() + 1e-30
    return out, lse, bound, dz + 2.0 ** -18 + 2.0 ** -21 * lse.abs()


def check(q, cache, scales, tables, lens, v_dim, scale, got, prefix=None, page=None):
    """got = (out, lse) of requests whose tokens are those of `prefix` (table,
    length) and then lens[b] of tables[b]."""
    out, lse = got
    page = page or cache.shape[1]
    K = 2 * q.shape[2] - cache.shape[2]
    v = values(cache, scales, K)
    codes = cache.contiguous()[..., :v_dim].contiguous().view(E4).double().abs().flatten(0, 1)
    s = scales.double().flatten()
    front = slots_of(prefix[0], page, 0, prefix[1]) if prefix else torch.empty(0, dtype=I64, device=DEV)
    for b, n in enumerate(lens):
        # Blocks of 32 begin anew behind the prefix: their largest weights bound more than one of both would.
        at = torch.cat([front, slots_of(tables[b], page, 0, n)])
        o, l, bound, dl = reference(q[b].double(), v[at], codes[at], s[at], scale, v_dim)
        err = (out[b].double() - o).abs()
        assert (err <= bound).all(), f"request {b}: {float((err / bound).max()):.2f} of the bound"
        if not at.numel():
            assert (lse[b] == -math.inf).all() and (out[b] == 0).all()
        else:
            assert ((lse[b].double() - l).abs() <= dl).all(), f"request {b}: lse off by {float((lse[b].double() - l).abs().max()):.2e}"


LONG = False                          # tables of many columns that no request uses


@pytest.fixture(params=["short tables", "long tables"])
def tables(request, monkeypatch):
    """Heads go to CTAs by 16 or 32 where the tables hold few tokens, by 64 otherwise."""
    monkeypatch.setattr(sys.modules[__name__], "LONG", request.param == "long tables")


both = pytest.mark.usefixtures("tables")


def paged(g, lens, page, spare=3, extra=2):
    held = [-(-n // page) for n in lens]
    if LONG:
        extra += 1300 * 128 // (max(len(lens), 1) * page)
    pages = sum(held) + spare
    ids = torch.randperm(pages, generator=g, device=DEV).to(I32)
    table = torch.full((len(lens), max(held, default=0) + extra), -1, dtype=I32, device=DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def spoil(cache, scales, table, lens, page):
    """NaN wherever no token lies: behind the last one of a page, and on spare pages."""
    used = torch.zeros(cache.shape[0] * page, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        used[slots_of(table[b], page, 0, n)] = True
    flat = cache.view(-1, cache.shape[-1])
    flat[~used] = 0xff
    scales.view(-1)[~used] = math.nan


def run(lens, H, K, P, DV, page, seed, spread=0.0, scale=None):
    g = gen(seed)
    table, pages = paged(g, lens, page)
    cache, scales = make_cache(g, pages, page, K, P, spread)
    spoil(cache, scales, table, lens, page)
    q = randn(g, len(lens), H, K + P)
    scale = scale or (K + P) ** -0.5 * 3
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), DV, scale)
    assert dsnq.debug_status() == OK
    clean = torch.nan_to_num(scales, nan=1.0)
    check(q, cache, clean, table, lens, DV, scale, got)
    return got


@both
@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 192, 256])
def test_attention_page_sizes(page):
    run([1, 0, 127, 300, 1000], 16, 512, 64, 512, page, seed=page)


@both
@pytest.mark.parametrize("H", [1, 2, 7, 8, 16, 17, 32, 33, 48, 63, 64, 65, 100, 128, 130, 200])
def test_attention_heads(H):
    run([5, 200, 129, 0], H, 512, 64, 512, 64, seed=H)


@both
@pytest.mark.parametrize("K,P,DV", [(128, 0, 128), (128, 64, 128), (256, 0, 128), (256, 64, 256), (384, 0, 384), (384, 64, 256), (512, 0, 512),
                                    (512, 64, 128), (512, 64, 512)])
@pytest.mark.parametrize("H", [5, 48, 64])
def test_attention_widths(K, P, DV, H):
    run([1, 64, 700, 1500, 260], H, K, P, DV, 32, seed=K + P + DV)


@both
def test_attention_lengths_around_every_tile_border():
    run([n for t in (32, 64, 96, 128, 256, 384) for n in (t - 1, t, t + 1)], 8, 512, 64, 512, 64, seed=1)


@both
@pytest.mark.parametrize("lens,H", [([20000], 16), ([9000, 3], 128), ([0, 5000, 0, 1], 64), ([1] * 400, 8), ([128] * 160 + [0] * 30, 65),
                                    ([3000] * 152, 16), ([2000] * 80, 128), ([40000], 64), (list(range(0, 3000, 37)), 48), ([0] * 9, 3)])
def test_attention_work_splits(lens, H):
    run(lens, H, 512, 64, 512, 64, seed=len(lens) + H)


@both
@pytest.mark.parametrize("K,P,H", [(512, 64, 16), (512, 64, 32), (512, 64, 48), (512, 64, 64), (512, 0, 48), (512, 0, 64), (384, 64, 64),
                                   (256, 64, 16), (128, 0, 64), (128, 64, 16)])
def test_attention_long_runs_of_every_ring(K, P, H):
    """Workers of many tiles: the rings of chunks go around many times."""
    run([30000, 11111], H, K, P, K, 16, seed=K + P + H)


@both
@pytest.mark.parametrize("spread", [2.0, 6.0])
def test_attention_scales_far_apart(spread):
    run([300, 90, 2000], 20, 256, 64, 256, 16, seed=5, spread=spread)


def test_attention_most_heads_requests_and_a_table_of_no_columns():
    run([3, 200], 1024, 128, 0, 128, 8, seed=2)
    run([n % 5 for n in range(8192)], 1, 128, 0, 128, 8, seed=3)
    cache, scales = make_cache(gen(1), 1, 8, 128, 0)
    out, lse = dsnq.paged_latent_attention_fp8(randn(gen(2), 3, 4, 128), cache, scales, torch.empty(3, 0, dtype=I32, device=DEV), ints([5, 0, 9]), 128, 1.0)
    assert (out == 0).all() and (lse == -math.inf).all() and dsnq.debug_status() == OK


@both
def test_attention_scores_that_grow_and_peak():
    """Scores that grow by hundreds from tile to tile (O and the sums follow),
    fall, and one token far above all others; a sink far above a long tail."""
    K, page = 128, 32
    for H, lens, shape in ((64, [1200, 2500], "grow"), (16, [1200, 2500], "fall"), (33, [900, 5000], "peak"), (16, [9000], "sink")):
        g = gen(H)
        table, pages = paged(g, lens, page)
        cache, scales = make_cache(g, pages, page, K, 0)
        q = randn(g, len(lens), H, K).abs() + 0.5
        for b, n in enumerate(lens):
            at = slots_of(table[b], page, 0, n)
            t = torch.arange(n, device=DEV, dtype=F32)
            level = {"grow": t / 3, "fall": (n - t) / 3, "peak": torch.where(t == n // 3, 300.0, 1.0),
                     "sink": torch.where(t == 0, 10.0, 0.02 * torch.rand(n, generator=g, device=DEV))}[shape]
            cache.view(-1, K)[at] = (torch.rand(n, K, generator=g, device=DEV) * 100 + 300).to(E4).view(U8)
            scales.view(-1)[at] = level.clamp(min=1e-3) / 400
        got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.02)
        check(q, cache, scales, table, lens, K, 0.02, got)
        assert dsnq.debug_status() == OK


@both
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("n", [1, 2, 31, 500])
def test_attention_of_equal_values_is_that_value(H, n):
    """The weights add up to one: whatever the scores, tokens with the same
    value give that value, to the bf16's own rounding."""
    K, P = 256, 64
    g = gen(n)
    table, pages = paged(g, [n], 16)
    cache, scales = make_cache(g, pages, 16, K, P)
    cache[..., :K] = cache[0, 0, :K]
    scales.fill_(0.0123)
    q = randn(g, 1, H, K + P)
    out, _ = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints([n]), K, 0.05)
    want = cache[0, 0, :K].view(E4).double() * float(scales[0, 0])
    assert ((out[0].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18)).all()


@both
def test_attention_rows_of_no_scale():
    """A scale of 0 (a row never written): a zero row, with the weight of a zero score."""
    g = gen(8)
    table, pages = paged(g, [40, 300], 8)
    cache, scales = make_cache(g, pages, 8, 128, 64)
    for b, n in ((0, 40), (1, 300)):
        scales.view(-1)[slots_of(table[b], 8, 0, n)[3::4]] = 0
    q = randn(g, 2, 9, 192)
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints([40, 300]), 128, 0.1)
    check(q, cache, scales, table, [40, 300], 128, 0.1, got)


@both
@pytest.mark.parametrize("H,K", [(20, 256), (64, 512)])
def test_attention_bad_pages_read_as_zero_rows_and_are_reported(H, K):
    g = gen(9)
    lens = [300, 70, 5]
    table, pages = paged(g, lens, 16)
    cache, scales = make_cache(g, pages, 16, K, 64)
    q = randn(g, 3, H, K + 64)
    good = table.clone()
    table[0, 3], table[0, 18], table[1, 0], table[2, 0] = pages, -5, 2 ** 31 - 1, -2 ** 31
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.1)
    assert dsnq.debug_status() == BOUNDS and dsnq.debug_status() == OK
    zeros = torch.zeros(1, 16, cache.shape[-1], dtype=U8, device=DEV)
    more, more_s = torch.cat([cache, zeros]), torch.cat([scales, torch.zeros(1, 16, device=DEV)])
    table = torch.where((table < 0) | (table >= pages), pages, table)
    table = torch.where(good < 0, good, table)
    check(q, more, more_s, table, lens, K, 0.1, got)


def test_attention_lengths_outside_the_table():
    g = gen(10)
    cache, scales = make_cache(g, 8, 16, 128, 0)
    table = ints([[0, 1], [2, 3], [4, 5]])
    q = randn(g, 3, 4, 128)
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints([33, -4, 2 ** 31 - 1]), 128, 0.2)
    check(q, cache, scales, table, [32, 0, 32], 128, 0.2, got)
    assert dsnq.debug_status() == OK


@both
def test_attention_strided_views():
    g = gen(11)
    lens, K, P, H = [200, 37, 130], 256, 64, 10
    table, pages = paged(g, lens, 16)
    big = torch.zeros(pages, 20, K + 2 * P + 48, dtype=U8, device=DEV)
    c0, s0 = make_cache(g, pages, 16, K, P)
    cache = big[:, 2:18, 16:16 + K + 2 * P]
    cache.copy_(c0)
    scales = torch.zeros(pages, 28, device=DEV)[:, 8:24]
    scales.copy_(s0)
    wide_q = randn(g, 3, H + 2, K + P + 8)
    q = wide_q[:, 1:H + 1, :K + P]
    wide_out = torch.full((3, H + 3, K + 16), 7.0, dtype=BF, device=DEV)
    wide_lse = torch.full((3, H + 5), 7.0, device=DEV)
    wide_table = torch.full((3, table.shape[1] + 4), -1, dtype=I32, device=DEV)
    wide_table[:, 3:3 + table.shape[1]] = table
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, wide_table[:, 3:3 + table.shape[1]], ints(lens), K, 0.1,
                                          out=wide_out[:, 2:H + 2, 8:K + 8], lse=wide_lse[:, 1:H + 1])
    check(q, c0, s0, table, lens, K, 0.1, got)
    wide_out[:, 2:H + 2, 8:K + 8] = 7
    wide_lse[:, 1:H + 1] = 7
    assert (wide_out == 7).all() and (wide_lse == 7).all()


@both
def test_attention_non_finite_queries_stay_in_their_heads():
    g = gen(12)
    lens, K, P = [300, 4000], 512, 64
    table, pages = paged(g, lens, 64)
    cache, scales = make_cache(g, pages, 64, K, P)
    for H in (16, 64):
        q = randn(g, 2, H, K + P)
        clean = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.1)
        bad = q.clone()
        bad[0, 3, 5], bad[1, 7, 100], bad[1, 0, K + 3] = math.nan, math.inf, math.nan
        out, lse = dsnq.paged_latent_attention_fp8(bad, cache, scales, table, ints(lens), K, 0.1)
        hit = torch.zeros(2, H, dtype=torch.bool, device=DEV)
        hit[0, 3] = hit[1, 7] = hit[1, 0] = True
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@both
@pytest.mark.parametrize("H", [3, 48, 64])
def test_attention_of_a_row_that_is_not_finite(H):
    """Its request is NaN in every head, the others are what they are without it."""
    g = gen(31)
    lens = [700, 90, 300]
    table, pages = paged(g, lens, 16)
    cache, scales = make_cache(g, pages, 16, 512, 64)
    q = randn(g, 3, H, 576)
    call = lambda: dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), 512, 0.05)
    want = call()
    scales.view(-1)[slots_of(table[1], 16, 33, 34)] = math.nan
    out, lse = call()
    assert out[1].isnan().all() and lse[1].isnan().all()
    for b in (0, 2):
        assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    assert dsnq.debug_status() == OK


@both
def test_attention_queries_of_any_size():
    """The split of q goes by each head's largest value: from 2^-90 to 2^90, and heads of zeros."""
    g = gen(13)
    lens = [200, 33]
    table, pages = paged(g, lens, 8)
    cache, scales = make_cache(g, pages, 8, 256, 64)
    for e in (-90, -20, 0, 20, 90):
        q = (randn(g, 2, 12, 320).float() * 2.0 ** e).to(BF)
        q[0, 3] = 0
        scale = 0.1 * 2.0 ** -e
        got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), 256, scale)
        check(q, cache, scales, table, lens, 256, float(np.float32(scale)), got)


@both
def test_attention_repeats_and_needs_no_clean_workspace():
    g = gen(14)
    lens = [5000, 3, 700, 128]
    table, pages = paged(g, lens, 64)
    cache, scales = make_cache(g, pages, 64, 512, 64)
    q = randn(g, 4, 16, 576)
    size = dsnq.paged_latent_attention_fp8_workspace_bytes(4, 16, 512, table.shape[1], 64)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((size,), fill, dtype=U8, device=DEV)
        got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), 512, 0.1, workspace=ws)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    with pytest.raises(dsnq.DsnqError):
        dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), 512, 0.1, workspace=ws[:-16])


def test_past_32_bit_offsets():
    """A cache of 5 GB: pages, rows and scales beyond 2^32 bytes."""
    K, P, page = 512, 64, 64
    pages = 5 * (1 << 30) // (page * (K + 2 * P)) + 1
    cache = torch.zeros(pages, page, K + 2 * P, dtype=U8, device=DEV)
    scales = torch.zeros(pages, page, device=DEV)
    g = gen(15)
    lens = [1000, 77]
    ids = torch.cat([torch.arange(pages - 10, pages, device=DEV), torch.arange(pages // 2, pages // 2 + 8, device=DEV)]).to(I32)
    table = torch.full((2, 16), -1, dtype=I32, device=DEV)
    table[0], table[1, :2] = ids[:16], ids[16:]
    M = sum(lens)
    slots = torch.cat([slots_of(table[b], page, 0, n) for b, n in enumerate(lens)])
    f, _ = dsnq.rope_frequencies(64, device=DEV)
    kv, pe = randn(g, M, K), randn(g, M, P)
    dsnq.latent_cache_write_fp8(kv, pe, torch.arange(M, device=DEV), slots, f, cache, scales)
    back = dsnq.latent_cache_read_fp8(cache, scales, K, table, ints([0, lens[0], M]), M)
    assert ((back[:, :K].float() - kv.float()).abs() <= kv.float().abs() * 2.0 ** -3.9 + 0.02).all()
    q = randn(g, 2, 16, K + P)
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.1)
    small_c, small_s = cache[ids.long()], scales[ids.long()]
    small_t = torch.full((2, 16), -1, dtype=I32, device=DEV)
    small_t[0], small_t[1, :2] = torch.arange(16, device=DEV).to(I32), torch.arange(16, 18, device=DEV).to(I32)
    check(q, small_c, small_s, small_t, lens, K, 0.1, got)
    assert dsnq.debug_status() == OK


# -------------------------------------------------------- behind a common prefix

def run_shared(prefix, lens, H, K, P, DV, page, seed, stored=None):
    g = gen(seed)
    table, pages = paged(g, [*lens, max(prefix, 0)], page)
    cache, scales = make_cache(g, pages, page, K, P)
    front = table[-1, :-(-max(prefix, 0) // page) + (stored is None)].contiguous()   # an entry that is not read, or none
    own = table[:-1].contiguous()
    spoil(cache, scales, table, [*lens, max(prefix, 0)], page)
    q = randn(g, len(lens), H, K + P)
    got = dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, front, ints([prefix if stored is None else stored]), own, ints(lens), DV, 0.1)
    assert dsnq.debug_status() == OK
    check(q, cache, torch.nan_to_num(scales, nan=1.0), own, lens, DV, 0.1, got, prefix=(front, max(prefix, 0)))
    return got


@both
@pytest.mark.parametrize("prefix", [0, 1, 31, 127, 128, 129, 1000, 5000])
@pytest.mark.parametrize("H", [1, 6, 16, 48, 64, 100, 128])
def test_shared_prefix(prefix, H):
    run_shared(prefix, [1, 0, 200, 129, 33], H, 512, 64, 512, 64, seed=prefix + H)


@both
@pytest.mark.parametrize("lens,H,prefix", [([0] * 7, 16, 300), ([0], 3, 0), ([5000, 1, 0], 16, 60), ([7] * 300, 8, 2000), ([100] * 160, 65, 129),
                                           ([64], 16, 20000), ([0, 0, 9000], 128, 9000), ([3] * 33, 200, 40)])
def test_shared_prefix_work_splits(lens, H, prefix):
    run_shared(prefix, lens, H, 512, 64, 512, 32, seed=len(lens))


@both
@pytest.mark.parametrize("K,P,DV,page", [(128, 0, 128, 8), (256, 64, 128, 48), (384, 64, 384, 128), (512, 0, 256, 16)])
def test_shared_prefix_widths(K, P, DV, page):
    run_shared(777, [50, 0, 300, 1], 24, K, P, DV, page, seed=K + P)


def test_shared_prefix_lengths_outside_its_table():
    """A prefix length past the table counts as the table's, a negative one as 0."""
    run_shared(256, [9, 100], 16, 128, 0, 128, 128, seed=1, stored=384)
    run_shared(0, [9, 100], 16, 128, 0, 128, 128, seed=1, stored=-5)


def test_shared_prefix_of_no_pages_and_bad_pages():
    g = gen(2)
    lens = [40, 3]
    table, pages = paged(g, lens, 8)
    cache, scales = make_cache(g, pages, 8, 128, 64)
    q = randn(g, 2, 5, 192)
    got = dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, torch.empty(0, dtype=I32, device=DEV), ints([70]), table, ints(lens), 128, 0.1)
    check(q, cache, scales, table, lens, 128, 0.1, got)
    assert dsnq.debug_status() == OK
    dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, ints([0, pages + 3]), ints([16]), table, ints(lens), 128, 0.1)
    assert dsnq.debug_status() == BOUNDS and dsnq.debug_status() == OK


@both
def test_shared_prefix_agrees_with_separate_requests():
    """The same tokens as requests of their own whose tables begin with the prefix's pages."""
    g = gen(3)
    lens, prefix, page, H = [70, 0, 300], 640, 64, 16
    table, pages = paged(g, [*lens, prefix], page)
    cache, scales = make_cache(g, pages, page, 512, 64)
    q = randn(g, 3, H, 576)
    front, own = table[-1, :10].contiguous(), table[:-1, :6].contiguous()
    a, la = dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, front, ints([prefix]), own, ints(lens), 512, 0.1)
    b, lb = dsnq.paged_latent_attention_fp8(q, cache, scales, torch.cat([front.expand(3, -1), own], 1), ints([prefix + n for n in lens]), 512, 0.1)
    # Two outputs within their bounds of the same values: 2^-8 of the weighted |values| and the output each, twice.
    top = (cache[..., :512].view(E4).float() * scales[..., None]).abs().max()
    assert ((a.float() - b.float()).abs() <= 4 * 2.0 ** -8 * top).all() and ((la - lb).abs() <= 2.0 ** -15).all()


@both
def test_shared_prefix_strides_repeats_and_workspaces():
    g = gen(4)
    lens, prefix, H = [70, 0, 300, 5], 700, 7
    table, pages = paged(g, [*lens, prefix], 16)
    cache, scales = make_cache(g, pages, 16, 256, 64)
    q = randn(g, 4, H + 1, 328)[:, 1:, :320]
    front, own = table[-1].contiguous(), table[:-1]
    out, lse = torch.full((4, H + 2, 264), 7.0, dtype=BF, device=DEV), torch.full((4, H + 1), 7.0, device=DEV)
    size = dsnq.shared_prefix_latent_attention_fp8_workspace_bytes(4, H, 256, front.numel(), own.shape[1], 16)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((size,), fill, dtype=U8, device=DEV)
        got = dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, front, ints([prefix]), own, ints(lens), 256, 0.1,
                                                      out=out[:, 1:H + 1, 8:], lse=lse[:, :H], workspace=ws)
        first = first or tuple(t.clone() for t in got)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    check(q, cache, scales, own, lens, 256, 0.1, first, prefix=(front, prefix))
    out[:, 1:H + 1, 8:] = 7
    assert (out == 7).all() and (lse[:, H] == 7).all()
    with pytest.raises(dsnq.DsnqError):
        dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, front, ints([prefix]), own, ints(lens), 256, 0.1, workspace=ws[:-16])


# ------------------------------------------------------------------ runs of them

def serving_step(s):
    """One step of a serving loop: pages, the write of the new tokens, attention
    behind the prefix."""
    lens, _, pos, slots, _ = dsnq.extend_block_tables(s["lens"], None, s["free"], s["table"], 16, s["B"])
    dsnq.latent_cache_write_fp8(s["kv"], s["pe"], pos + s["prefix"], slots, s["freq"], s["cache"], s["scales"], normalize=True)
    q = dsnq.head_rmsnorm_rope(s["q"], pos + s["prefix"], s["freq"], normalize=False)
    return (lens, *dsnq.shared_prefix_latent_attention_fp8(q, s["cache"], s["scales"], s["front"], s["prefix_len"], s["table"], lens, 512, 0.08))


def serving_state(seed, B=9, H=16, prefix=200):
    g = gen(seed)
    s = dict(B=B, prefix=prefix, lens=torch.randint(0, 60, (B,), generator=g, device=DEV).to(I32), kv=randn(g, B, 512), pe=randn(g, B, 64),
             q=randn(g, B, H, 576), prefix_len=ints([prefix]), freq=dsnq.rope_frequencies(64, device=DEV)[0])
    s["cache"], s["scales"] = make_cache(g, 100, 16, 512, 64)
    ids = torch.randperm(100, generator=g, device=DEV).to(I32)
    s["front"], s["free"] = ids[:13].clone(), ids[13 + 4 * B:].clone()
    s["table"] = torch.full((B, 6), -1, dtype=I32, device=DEV)
    s["table"][:, :4] = ids[13:13 + 4 * B].view(B, 4)
    return s


def test_serving_step_and_its_graph():
    s, t = serving_state(1), serving_state(1)
    before = s["lens"].tolist()
    lens, out, lse = serving_step(s)
    assert lens.tolist() == [n + 1 for n in before] and dsnq.debug_status() == OK
    pos = ints(before).long() + s["prefix"]
    q = dsnq.head_rmsnorm_rope(s["q"], pos, s["freq"], normalize=False)
    check(q, s["cache"], s["scales"], s["table"], lens.tolist(), 512, float(np.float32(0.08)), (out, lse), prefix=(s["front"], s["prefix"]))
    serving_step(t)                                            # (the kernels are loaded)
    t = serving_state(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = serving_step(t)
    fresh = serving_state(1)
    for k in ("cache", "scales", "table"):
        t[k].copy_(fresh[k])
    for _ in range(2):                                         # the same step again: the same outputs
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, (lens, out, lse)):
            assert torch.equal(a, b)


def test_two_graphs_and_two_streams_at_once():
    states = [serving_state(i, B=20 + i, prefix=1500) for i in range(2)]
    want = [serving_step(serving_state(i, B=20 + i, prefix=1500)) for i in range(2)]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(serving_step(s))
        graphs.append(graph)
    for i, fresh in enumerate(serving_state(i, B=20 + i, prefix=1500) for i in range(2)):
        for k in ("cache", "scales", "table"):
            states[i][k].copy_(fresh[k])
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # Eager calls on two streams, each with the workspace of its own stream.
    results = [None, None]
    fresh = [serving_state(i, B=20 + i, prefix=1500) for i in range(2)]
    torch.cuda.synchronize()
    for i, stream in enumerate(streams):
        with torch.cuda.stream(stream):
            results[i] = serving_step(fresh[i])
    torch.cuda.synchronize()
    for a, b in zip(results, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert dsnq.debug_status() == OK


def test_explicit_stream():
    s = serving_state(5)
    want = serving_step(serving_state(5))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    lens, _, pos, slots, _ = dsnq.extend_block_tables(s["lens"], None, s["free"], s["table"], 16, s["B"], stream=stream)
    with torch.cuda.stream(stream):
        pos = pos + s["prefix"]
    dsnq.latent_cache_write_fp8(s["kv"], s["pe"], pos, slots, s["freq"], s["cache"], s["scales"], normalize=True, stream=stream)
    q = dsnq.head_rmsnorm_rope(s["q"], pos, s["freq"], normalize=False, stream=stream)
    out, lse = dsnq.shared_prefix_latent_attention_fp8(q, s["cache"], s["scales"], s["front"], s["prefix_len"], s["table"], lens, 512, 0.08,
                                                       stream=stream)
    rows = dsnq.latent_cache_read_fp8(s["cache"], s["scales"], 512, s["table"], ints([0] + [0] * s["B"]), 4, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want[1]) and torch.equal(lse, want[2]) and rows.shape == (4, 576)


@pytest.mark.parametrize("page", [16, 64])
def test_wait_runs_out_and_is_reported(page):
    """The first copy never comes: the kernel gives up after the limit, reports
    it, and the next call is as ever."""
    g = gen(6)
    lens = [700, 300]
    table, pages = paged(g, lens, page)
    cache, scales = make_cache(g, pages, page, 512, 64)
    q = randn(g, 2, 64, 576)
    call = lambda: dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), 512, 0.1)
    want = call()
    torch.cuda.synchronize()
    try:
        dsnq.debug_set(1, 20_000_000)
        call()
        assert dsnq.debug_status() == TIMEOUT
    finally:
        dsnq.debug_set(0, 0)
    got = call()
    assert dsnq.debug_status() == OK and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_launch_overlap_changes_nothing():
    want = serving_step(serving_state(7))
    try:
        dsnq.set_launch_overlap(False)
        got = serving_step(serving_state(7))
    finally:
        dsnq.set_launch_overlap(True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_requests():
    cache, scales = make_cache(gen(1), 2, 8, 128, 64)
    empty = torch.empty(0, 2, dtype=I32, device=DEV)
    out, lse = dsnq.paged_latent_attention_fp8(torch.empty(0, 4, 192, dtype=BF, device=DEV), cache, scales, empty, ints([]), 128, 1.0)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    out, lse = dsnq.shared_prefix_latent_attention_fp8(torch.empty(0, 4, 192, dtype=BF, device=DEV), cache, scales, ints([0]), ints([5]), empty,
                                                       ints([]), 128, 1.0)
    assert out.shape == (0, 4, 128)
    dsnq.latent_cache_write_fp8(torch.empty(0, 128, dtype=BF, device=DEV), torch.empty(0, 64, dtype=BF, device=DEV),
                                torch.empty(0, dtype=I64, device=DEV), torch.empty(0, dtype=I64, device=DEV),
                                torch.empty(32, dtype=F64, device=DEV), cache, scales)
    assert dsnq.debug_status() == OK


@both
@pytest.mark.parametrize("size", [0.0, 2.0 ** -90, 2.0 ** -20, 1.0])
@pytest.mark.parametrize("H", [9, 64])
def test_attention_of_queries_in_the_position_columns(H, size):
    """Latent columns of q that are zero or far below its position columns, over
    rows whose latent is zero or tiny, so that the cache holds position columns
    of up to 2^61 (pe / s).  Scores and weights are those of ordinary numbers."""
    K, P, page = 256, 64, 16
    g = gen(H)
    lens = [150, 700]
    table, pages = paged(g, lens, page)
    cache, scales = make_cache(g, pages, page, K, P)
    for b, n in enumerate(lens):
        at = slots_of(table[b], page, 0, n)
        level = torch.tensor([0.0, 2.0 ** -33, 2.0 ** -13, 1.0], device=DEV)[torch.arange(n, device=DEV) % 4]
        dsnq.latent_cache_write_fp8((torch.randn(n, K, generator=g, device=DEV) * level[:, None]).to(BF), randn(g, n, P),
                                    torch.zeros(n, dtype=I64, device=DEV), at, torch.empty(0, dtype=F64, device=DEV), cache, scales)
    assert scales.min() == 2.0 ** -60
    q = torch.cat([(torch.randn(2, H, K, generator=g, device=DEV) * size).to(BF), randn(g, 2, H, P)], -1)
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.1)
    check(q, cache, scales, table, lens, K, float(np.float32(0.1)), got)
    front = table[1, :-(-700 // page)].contiguous()
    got = dsnq.shared_prefix_latent_attention_fp8(q[:1], cache, scales, front, ints([700]), table[:1], ints([150]), K, 0.1)
    check(q[:1], cache, scales, table[:1], [150], K, float(np.float32(0.1)), got, prefix=(front, 700))
    assert dsnq.debug_status() == OK


@both
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_of_scores_near_the_end_of_fp32(H, sign):
    """Scores of 2^104 in magnitude, all tokens alike: masked tokens stay below
    the lowest of them, and the output is the tokens' value."""
    K, page = 256, 16
    g = gen(H)
    lens = [1, 33, 500]
    table, pages = paged(g, lens, page)
    cache, scales = make_cache(g, pages, page, K, 0)
    cache[:] = cache[0, 0]
    scales.fill_(0.0123)
    code = cache[0, 0].view(E4).double()
    q = (sign * code.sign() * 2.0 ** 100).to(BF).expand(3, H, K).contiguous()
    out, lse = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.05)
    want = code * float(scales[0, 0])
    assert ((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
    score = sign * 2.0 ** 100 * code.abs().sum() * float(scales[0, 0]) * float(np.float32(0.05))
    # Products of a power of two and few bits; what is left are the sum's truncations (dz) and six roundings.
    assert ((lse.double() - score).abs() <= (K / 32 + 8) * 2.0 ** -23 * abs(score)).all()
    assert dsnq.debug_status() == OK


@both
@pytest.mark.parametrize("H", [16, 64])
def test_attention_scales_at_the_ends_of_their_range(H):
    """Scales of one request 2^80 apart, from an all-zero row's on: rows of the
    smallest scale count with their probability, whatever the others hold."""
    K, page = 128, 16
    g = gen(H)
    lens = [300, 40, 1500]
    table, pages = paged(g, lens, page)
    cache, scales = make_cache(g, pages, page, K, 0)
    for b, n in enumerate(lens):
        at = slots_of(table[b], page, 0, n)
        which = torch.randint(0, 3, (n,), generator=g, device=DEV)
        which = torch.where(torch.arange(n, device=DEV) // 64 % 3 == 2, 0, which)       # whole blocks of the smallest too
        scales.view(-1)[at] = torch.tensor([2.0 ** -60, 2.0 ** -8, 2.0 ** 20], device=DEV)[which]
    q = (torch.randn(3, H, K, generator=g, device=DEV) * 2.0 ** -29).to(BF)
    got = dsnq.paged_latent_attention_fp8(q, cache, scales, table, ints(lens), K, 0.1)
    check(q, cache, scales, table, lens, K, float(np.float32(0.1)), got)
    assert dsnq.debug_status() == OK
