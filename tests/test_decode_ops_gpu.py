"""The decode-step operators on the GPU against their fp64 oracle: block
tables, head norm + rotary, latent cache write, paged latent attention, and a
run of them behind the pre-projection.

Tolerances.  A result is rounded once to bf16: half a step, 2^-8 of the value
at most.  Rotation: the fp32 arithmetic before the rounding (norm: a sum over
at most 1024 values, so a relative 2^-15 covers its 1024 * 2^-24 / 2 and the
square root; cos, sin and two products: 2^-21) acts on the pair, so it is
bounded by 2^-14 of |a| + |b|.  Attention: each probability is rounded to bf16
(2^-8) before the product with the values, and a score is off by at most dz =
(DK/16 + 4) * 2^-23 of the largest sum of |q k| * scale (one fp32 addition per
16-wide step of the tensor core, whose additions truncate), which moves every
probability by 2 dz relative; sums and exponentials add 2^-18.  So an output
is within (2^-8 + 2 dz + 2^-18) sum p |v| + 2^-8 |out|, and lse within dz +
2^-20 + 2^-21 |lse|."""

import numpy as np
import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq
import oracle
from gemm_dsnq_dual_gb300 import inputs

pytestmark = pytest.mark.gpu
OK, TIMEOUT, BOUNDS = 0, 5, 6
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def val(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- block tables

def check_extend(lens, new, free, table, page, rows, out=None):
    ref = oracle.extend_block_tables(lens, new, free, table, page, rows)
    t = torch.tensor(table, dtype=torch.int32, device=DEV).reshape(len(lens), -1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    got = dsnq.extend_block_tables(i32(lens), None if new is None else i32(new), i32(free), t, page, rows, out=out)
    names = ("new_lens", "row_starts", "positions", "slots", "counts", "table")
    for name, g, r in zip(names, (*got, t), ref):
        assert np.array_equal(g.cpu().numpy(), r.reshape(g.shape)), name
    assert dsnq.debug_status() == OK


def extend_case(B, page, seed, most=300, prompts=True):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most, B)
    lens[rng.random(B) < 0.15] = 0
    new = np.ones(B, np.int64)
    if prompts:
        pick = rng.random(B) < 0.3
        new[pick] = rng.integers(0, 3 * page + 5, pick.sum())
    width = int((lens + new).max() // page + 2)
    held = -(-lens // page)
    pool = rng.permutation(int(held.sum()) + 500)
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    need = int((-(-(lens + new) // page) - held).sum())
    return lens, new, pool[at:at + need + 3], table, need


@pytest.mark.parametrize("page", [1, 8, 13, 64])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 257, 513, 1300])
def test_extend(B, page):
    lens, new, free, table, _ = extend_case(B, page, seed=B * 100 + page)
    check_extend(lens, new, free, table, page, int(new.sum()) + B % 5)


def test_extend_one_token_each():
    lens, _, free, table, _ = extend_case(70, 16, seed=3, prompts=False)
    check_extend(lens, None, free, table, 16, 70)
    check_extend(lens, None, free, table, 16, 64)            # the last six have no row
    check_extend(lens, None, free, table, 16, 0)


def test_extend_short_of_pages_rows_and_table():
    lens, new, free, table, need = extend_case(90, 8, seed=4)
    for n in (0, 1, need // 2, need - 1):
        check_extend(lens, new, free[:n], table, 8, int(new.sum()))
    check_extend(lens, new, free, table, 8, int(new.sum()) // 2)
    check_extend(lens, new, free, table[:, :10], 8, int(new.sum()) + 7)     # lengths beyond the table


def test_extend_odd_lengths():
    """Negative lengths and counts, a length past the table, empty counts."""
    table = np.arange(20).reshape(5, 4)
    check_extend([-3, 0, 16, 99, 7], [2, -1, 1, 3, 0], [50, 51, 52], table, 4, 9)
    check_extend([1, 2, 3, 4, 5], [0, 0, 0, 0, 0], [], table, 4, 3)


def test_extend_a_page_id_that_is_none():
    """A held page or a listed page with a negative id gives no slot."""
    check_extend([5, 4], [2, 1], [-1], np.array([[3, -1, 9], [8, -1, -1]]), 4, 3)


def test_extend_large_prompt_and_largest_batch():
    lens, new, free, table, need = extend_case(6, 16, seed=6)
    new[3] = 40000
    width = int((lens + new).max() // 16 + 2)
    t = np.full((6, width), -1)
    t[:, :table.shape[1]] = table
    held = -(-lens // 16)
    need = int((-(-(lens + new) // 16) - held).sum())
    check_extend(lens, new, np.arange(10000, 10000 + need), t, 16, int(new.sum()))
    for B in (2047, 2049, 4097):                             # around where the sums outgrow 32 and 48 KB
        t = np.arange(2 * B).reshape(B, 2)
        check_extend(np.arange(B) % 13, None, [], t, 16, B)
    B = 8192
    lens = np.arange(B) % 33
    t = np.full((B, 4), -1)
    t[:, :2] = np.arange(2 * B).reshape(B, 2)
    t[lens > 32, 2] = 7
    check_extend(lens, None, np.arange(50000, 50000 + B), t, 16, B)


def test_extend_strided_table_and_untouched_entries():
    """A table inside a wider buffer; entries of no new page keep their value."""
    buf = torch.full((3, 12), -99, dtype=torch.int32, device=DEV)
    table = buf[:, 2:7]
    table[:, 0] = torch.tensor([4, 5, 6], device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    dsnq.extend_block_tables(i32([3, 4, 1]), i32([1, 1, 9]), i32([11, 12, 13, 14]), table, 4, 11)
    want = np.full((3, 12), -99)
    want[:, 2] = [4, 5, 6]
    want[1, 3], want[2, 3:5] = 11, [12, 13]
    assert np.array_equal(buf.cpu().numpy(), want)


def test_extend_no_requests():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    lens, starts, pos, slots, counts = dsnq.extend_block_tables(e, None, e, torch.empty(0, 3, dtype=torch.int32, device=DEV), 16, 5)
    assert lens.numel() == 0 and starts.tolist() == [0] and counts.tolist() == [0, 0]
    assert pos.tolist() == [0] * 5 and slots.tolist() == [-1] * 5


# ---------------------------------------------------------- head norm + rotary

def check_rope(x, pos, f, out=None, **kw):
    D, R = x.shape[-1], 2 * len(f)
    off = kw.pop("rope_offset", D - R)
    gamma, norm, layout = kw.get("gamma"), kw.get("normalize", True), kw.get("layout", "interleaved")
    plain = oracle.head_rmsnorm_rope(val(x), pos.tolist(), f.tolist(), None if gamma is None else val(gamma), kw.get("eps", 1e-6),
                                     norm, off, layout, kw.get("rope_scale", 1.0), kw.get("inverse", False))
    still = oracle.head_rmsnorm_rope(val(x), pos.tolist(), [], None if gamma is None else val(gamma), kw.get("eps", 1e-6), norm, off)
    pair = np.abs(still)
    if R:
        v = np.abs(still[..., off:off + R])
        both = v[..., 0::2] + v[..., 1::2] if layout == "interleaved" else v[..., :R // 2] + v[..., R // 2:]
        pair[..., off:off + R] = abs(kw.get("rope_scale", 1.0)) * (
            np.repeat(both, 2, -1) if layout == "interleaved" else np.concatenate([both, both], -1))
    got = dsnq.head_rmsnorm_rope(x, pos, f, rope_offset=off, out=out, **kw)
    bound = 2.0 ** -8 * np.abs(plain) + 2.0 ** -14 * pair + 1e-38
    assert np.all(np.abs(val(got) - plain) <= bound), float(np.max(np.abs(val(got) - plain) / bound))
    assert dsnq.debug_status() == OK
    return got


FREQ = lambda R: dsnq.rope_frequencies(R)[0] if R else torch.empty(0, dtype=torch.float64, device=DEV)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,H,D,R,off", [
    (1, 1, 8, 0, 0), (1, 128, 192, 64, 128), (2, 3, 64, 64, 0), (3, 5, 72, 16, 24), (7, 32, 128, 64, 64), (5, 9, 136, 32, 8),
    (2, 48, 512, 64, 448), (3, 7, 264, 64, 96), (2, 11, 576, 64, 512), (2, 3, 1024, 256, 768), (1, 4, 520, 256, 120),
    (600, 17, 128, 32, 96), (1300, 3, 192, 64, 128)])
def test_head_norm_rope(M, H, D, R, off, layout):
    g = gen(M * 7 + D)
    x = randn(g, M, H, D)
    pos = torch.randint(0, 100000, (M,), generator=g, device=DEV)
    gamma = (torch.rand(D, generator=g, device=DEV) + 0.5).to(torch.bfloat16)
    f = FREQ(R)
    check_rope(x, pos, f, rope_offset=off, layout=layout, gamma=gamma)
    check_rope(x, pos, f, rope_offset=off, layout=layout)
    check_rope(x, pos, f, rope_offset=off, layout=layout, normalize=False, rope_scale=1.25)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_far_and_negative_positions(layout):
    """Angles of positions up to 2^31, where an fp32 angle would be noise.
    (The oracle's fp64 angle is itself off by 2^31 * 2^-53 rad there.)"""
    g = gen(1)
    pos = torch.tensor([0, 1, -1, -4096, 4097, 999983, 10 ** 6, 123456789, 2 ** 31 - 1, 2 ** 31], device=DEV)
    check_rope(randn(g, 10, 4, 64), pos, FREQ(64), layout=layout, normalize=False)
    f, s = dsnq.rope_frequencies(64, base=500000.0, factor=8.0, original_length=8192)
    check_rope(randn(g, 10, 4, 192), pos, f, layout=layout, rope_scale=s)


def test_frequencies_of_any_table():
    """Zero, negative and more than one turn per position."""
    g = gen(2)
    f = torch.tensor([0.0, -0.5, 7.25, 1e-9, 6.283185307179586, 3.0, 100.0, 1.0], dtype=torch.float64, device=DEV)
    check_rope(randn(g, 50, 2, 16), torch.arange(50, device=DEV), f, normalize=False)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("D,R", [(192, 64), (512, 256), (1024, 128), (64, 64)])
def test_rope_in_place_and_back(layout, D, R):
    g = gen(3)
    x = randn(g, 37, 19, D)
    pos = torch.randint(0, 5000, (37,), generator=g, device=DEV)
    want = dsnq.head_rmsnorm_rope(x, pos, FREQ(R), normalize=False, layout=layout)
    y = x.clone()
    got = dsnq.head_rmsnorm_rope(y, pos, FREQ(R), normalize=False, layout=layout, out=y)
    assert got is y and torch.equal(y, want)
    check_rope(y, pos, FREQ(R), normalize=False, layout=layout, inverse=True)


def test_rope_strided_views():
    """Heads inside a wider projection row, the output inside the queries of
    the attention; nothing else is written."""
    g = gen(4)
    row = randn(g, 9, 5 * 192 + 64)
    x = row[:, :5 * 192].view(9, 5, 192)
    pos = torch.arange(9, device=DEV)
    q = torch.full((9, 5, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    check_rope(x[:, :, 128:], pos, FREQ(64), out=q[:, :, 512:], normalize=False)
    assert bool((q[:, :, :512] == 7).all())
    t = randn(g, 5, 9, 128).transpose(0, 1)                  # heads outermost in memory
    check_rope(t, pos, FREQ(32))
    one = randn(g, 1, 1, 64)
    check_rope(one, pos[:1], FREQ(64))


def test_rope_zero_rows_and_non_finite():
    """A zero row stays zero (eps), an infinity or NaN stays in its own head."""
    g = gen(5)
    x = randn(g, 3, 4, 64)
    x[1, 2] = 0
    y = check_rope(x, torch.arange(3, device=DEV), FREQ(64))
    assert bool((y[1, 2] == 0).all())
    x[0, 1, 5], x[2, 3, 60] = float("inf"), float("nan")
    z = dsnq.head_rmsnorm_rope(x, torch.arange(3, device=DEV), FREQ(64))
    keep = torch.ones(3, 4, dtype=torch.bool, device=DEV)
    keep[0, 1] = keep[2, 3] = False
    assert torch.equal(z[keep], y[keep]) and not bool(torch.isfinite(z[2, 3]).any())


def test_rope_frequencies_of_every_size():
    """Zero, subnormal, tiny, negative and large frequencies against exact
    fractions of a turn.  The 64-bit step is off by |f| + 1 units of 2^-64
    turns, the turn by that times the position: 2^-21 turns at 2^30 and 5000,
    so 2^-18 rad beside the fp32 and bf16 steps of the other tests."""
    from fractions import Fraction
    per_turn = Fraction("0.159154943091895335768883763372514362034459645740456448747667344")   # 1 / (2 pi)
    f = [0.0, 5e-324, 1e-300, 2.0**-64, -2.0**-40, 1e-5, 0.3, -0.7, 1.0, 6.28318530717958, 33.3, -1000.1, 2.0**20 + 0.1,
         -(2.0**30), 2.0**30 - 0.5, 0.75]
    pos = [0, 1, 4999, -3]
    x = torch.zeros(len(pos), 2, 32, dtype=torch.bfloat16, device=DEV)
    x[:, 0, 0::2] = 1
    x[:, 1, 1::2] = 1
    got = val(dsnq.head_rmsnorm_rope(x, torch.tensor(pos, device=DEV), torch.tensor(f, dtype=torch.float64, device=DEV),
                                     normalize=False))
    t = np.array([[float((p * Fraction(w) * per_turn) % 1) for w in f] for p in pos]) * 2 * np.pi
    want = np.stack([np.stack([np.cos(t), np.sin(t)], -1), np.stack([-np.sin(t), np.cos(t)], -1)], 1).reshape(got.shape)
    assert np.all(np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-18 + 2.0**-14)


def test_rope_no_tokens():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert dsnq.head_rmsnorm_rope(e, torch.empty(0, dtype=torch.int64, device=DEV), FREQ(64)).shape == (0, 4, 64)


# ------------------------------------------------------------- cache write

@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,K,P,R,off,page", [
    (1, 512, 64, 64, 512, 64), (5, 512, 0, 64, 448, 16), (33, 256, 64, 64, 256, 1), (130, 8, 8, 0, 0, 3), (70, 512, 64, 128, 448, 64),
    (9, 960, 64, 256, 768, 5), (700, 128, 128, 32, 40, 128), (3, 768, 0, 16, 0, 7)])
def test_cache_write(M, K, P, R, off, page, layout):
    g = gen(M + K)
    buf = randn(g, M, 1536 + K + P + 8)
    kv, pe = buf[:, 1536:1536 + K], (buf[:, 1536 + K:1536 + K + P] if P else None)
    pages = -(-M // page) + 2
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:M]
    if M > 4:
        slots[3] = -1
        slots[M - 1] = -5
    pos = torch.randint(0, 1 << 20, (M,), generator=g, device=DEV)
    gamma = (torch.rand(K, generator=g, device=DEV) + 0.5).to(torch.bfloat16)
    f = FREQ(R)
    for norm, w in ((False, None), (True, None), (True, gamma)):
        wide = randn(g, pages, page, K + P + 16)             # rows inside wider ones
        before = wide.clone()
        cache = wide[:, :, 8:8 + K + P]
        assert dsnq.latent_cache_write(kv, pe, pos, slots, f, cache, gamma=w, normalize=norm, rope_offset=off, layout=layout,
                                       rope_scale=0.75) is cache
        a = (val(kv), None if pe is None else val(pe), pos.tolist())
        kw = dict(gamma=None if w is None else val(w), normalize=norm, rope_offset=off, layout=layout)
        ref = oracle.latent_rows(*a, f.tolist(), rope_scale=0.75, **kw)
        pair = np.abs(oracle.latent_rows(*a, [], **kw))
        if R:
            v = pair[:, off:off + R].copy()
            both = v[:, 0::2] + v[:, 1::2] if layout == "interleaved" else v[:, :R // 2] + v[:, R // 2:]
            pair[:, off:off + R] = np.repeat(both, 2, -1) if layout == "interleaved" else np.concatenate([both, both], -1)
        keep = (slots >= 0).cpu().numpy()
        got = val(cache.reshape(-1, K + P)[slots[slots >= 0]])
        bound = 2.0 ** -8 * np.abs(ref[keep]) + 2.0 ** -14 * pair[keep] + 1e-38
        assert np.all(np.abs(got - ref[keep]) <= bound)
        # Nothing else changed.
        mask = torch.zeros(pages * page, dtype=torch.bool, device=DEV)
        mask[slots[slots >= 0]] = True
        assert torch.equal(wide.reshape(pages * page, -1)[~mask], before.reshape(pages * page, -1)[~mask])
        assert torch.equal(wide[..., :8], before[..., :8]) and torch.equal(wide[..., -8:], before[..., -8:])
        assert dsnq.debug_status() == OK


def test_cache_write_reports_a_slot_past_the_cache():
    g = gen(6)
    kv, cache = randn(g, 3, 64), randn(g, 2, 8, 64)
    before = cache.clone()
    pos = torch.zeros(3, dtype=torch.int64, device=DEV)
    dsnq.latent_cache_write(kv, None, pos, torch.tensor([3, 16, 2 ** 40], device=DEV), FREQ(0), cache)
    assert dsnq.debug_status() == BOUNDS and dsnq.debug_status() == OK
    assert torch.equal(cache[0, 3], kv[0])
    cache[0, 3] = before[0, 3]
    assert torch.equal(cache, before)


def test_cache_write_and_attention_past_32_bit_offsets():
    """A cache of more than 2^32 elements (9.4 GB): a request whose rows lie
    at its end."""
    g = gen(7)
    pages = 130000
    cache = torch.empty(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    assert cache.numel() > 2 ** 32
    ids = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    n = 150
    kv, pe = randn(g, n, 512), randn(g, n, 64)
    j = torch.arange(n, device=DEV)
    slots = ids[0].long()[j // 64] * 64 + j % 64
    f = FREQ(64)
    dsnq.latent_cache_write(kv, pe, j, slots, f, cache)
    rows = oracle.latent_rows(val(kv), val(pe), j.tolist(), f.tolist(), rope_offset=512)
    got = val(cache.view(-1, 576)[slots])
    assert np.all(np.abs(got - rows) <= 2.0 ** -8 * np.abs(rows) + 2.0 ** -14 * 12)
    q = randn(g, 1, 16, 576)
    small = cache.view(-1, 576)[slots].clone()
    packed = torch.zeros(3, 64, 576, dtype=torch.bfloat16, device=DEV)
    packed.view(-1, 576)[:n] = small
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    a = dsnq.paged_latent_attention(q, cache, ids, lens, 512, 0.07)
    b = dsnq.paged_latent_attention(q, packed, torch.arange(3, dtype=torch.int32, device=DEV)[None], lens, 512, 0.07)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert dsnq.debug_status() == OK


# -------------------------------------------------------------- attention

def attention_case(lens, H, DK, page, seed, spare=3, extra=2, poison=True):
    """q, cache, table, lens.  Unused pages, the rows past a length and the
    table's unused entries hold garbage (NaN, infinities, wild ids)."""
    g = gen(seed)
    held = [-(-n // page) for n in lens]
    pool = torch.randperm(sum(held) + spare, generator=g, device=DEV).tolist()
    width = max(held + [0]) + extra
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32)
    cache = randn(g, sum(held) + spare, page, DK)
    if poison:
        used = torch.zeros(cache.shape[0], page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        mine = pool[at:at + held[b]]
        at += held[b]
        table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
        if poison:
            for k, p in enumerate(mine):
                used[p, :min(page, n - k * page)] = True
    if poison:
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38]).to(torch.bfloat16).to(DEV)
        junk = ~used.to(DEV)
        cache[junk] = bad[torch.randint(0, 4, (int(junk.sum()), DK), generator=g, device=DEV)]
    return randn(g, len(lens), H, DK), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def check_attention(q, cache, table, lens, DV, scale, ref=None, **kw):
    out, lse = dsnq.paged_latent_attention(q, cache, table, lens, DV, scale, **kw)
    assert dsnq.debug_status() == OK
    DK = q.shape[-1]
    if ref is None:
        ref = oracle.paged_latent_attention(val(q), val(cache), table.cpu().numpy(), lens.tolist(), DV, scale)
    want, want_lse, weight, reach = ref
    dz = (DK // 16 + 4) * 2.0 ** -23 * reach[..., None]
    bound = (2.0 ** -8 + 2 * dz + 2.0 ** -18) * weight + 2.0 ** -8 * np.abs(want) + 1e-38
    err = np.abs(val(out) - want)
    assert np.all(err <= bound), float(np.max(err / bound))
    empty = np.isinf(want_lse)
    assert np.array_equal(val(lse)[empty], want_lse[empty])
    got_lse, want_lse = val(lse)[~empty], want_lse[~empty]
    assert np.all(np.abs(got_lse - want_lse) <= dz[..., 0][~empty] + 2.0 ** -20 + 2.0 ** -21 * np.abs(want_lse))
    return out, lse


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 192])
def test_attention_page_sizes(page):
    lens = [1, page, page + 1, 63, 64, 65, 0, 129, 300]
    check_attention(*attention_case(lens, 20, 576, page, seed=page), 512, 576 ** -0.5)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 15, 16, 17, 48, 63, 64, 65, 100, 128, 130, 200])
def test_attention_heads(H):
    check_attention(*attention_case([130, 1, 0, 70], H, 576, 64, seed=H), 512, 0.05)


@pytest.mark.parametrize("DK,DV", [(128, 128), (192, 128), (256, 128), (256, 256), (320, 256), (448, 384), (512, 128), (512, 512),
                                   (576, 128), (576, 512)])
def test_attention_widths(DK, DV):
    check_attention(*attention_case([200, 64, 1, 129], 24, DK, 32, seed=DK + DV), DV, DK ** -0.5)


def test_attention_lengths_around_every_tile_border():
    lens = [n for t in (1, 2, 3, 5) for n in (64 * t - 1, 64 * t, 64 * t + 1)] + [0, 0, 2, 31, 33]
    check_attention(*attention_case(lens, 12, 576, 16, seed=9), 512, 0.06)


@pytest.mark.parametrize("lens,H", [([20000], 16), ([9000, 3], 128), ([0, 5000, 0, 1], 64), ([1] * 400, 8), ([64] * 160 + [0] * 30, 65),
                                    ([700] * 3 + [10000] + [5] * 40, 128), ([0] * 5, 128), ([0], 1),
                                    ([600, 590, 0, 610] * 17, 128), ([300] * 16, 64), ([130, 0, 1] * 50, 16)])
def test_attention_work_splits(lens, H):
    """One request over every worker, many to a worker, empty ones between."""
    check_attention(*attention_case(lens, H, 576, 64, seed=len(lens)), 512, 576 ** -0.5)


def test_attention_most_heads_requests_and_a_table_of_no_columns():
    """The largest batch and head count taken, no requests, no columns."""
    check_attention(*attention_case([70, 0, 3], 1024, 128, 8, seed=60), 128, 0.1)
    check_attention(*attention_case([5, 64], 513, 192, 64, seed=61), 128, 0.1)
    check_attention(*attention_case([k % 4 for k in range(8192)], 3, 128, 8, seed=62, poison=False), 128, 0.1)
    q, cache, table, lens = attention_case([9, 9], 20, 576, 64, seed=63)
    out, lse = dsnq.paged_latent_attention(q, cache, table[:, :0], lens, 512, 0.05)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    out, lse = dsnq.paged_latent_attention(q[:0], cache, table[:0], lens[:0], 512, 0.05)
    assert out.shape == (0, 20, 512) and lse.shape == (0, 20)
    assert dsnq.debug_status() == OK


@pytest.mark.parametrize("DK,DV", [(128, 128), (192, 128), (576, 128), (512, 256)])
def test_attention_long_narrow_rows(DK, DV):
    """Many tiles in the ring (narrow rows), and pairs of chunks that hold no value."""
    check_attention(*attention_case([7000, 130], 20, DK, 32, seed=DK), DV, DK ** -0.5)


def test_attention_no_request_sees_all_of_a_wide_table():
    """A table much wider than the lengths: idle workers."""
    check_attention(*attention_case([100, 5], 16, 576, 64, seed=10, extra=500), 512, 0.05)


def test_attention_scores_that_grow_and_peak():
    """The running maximum rises in every tile (keys in the order of their
    score), falls, and one key takes all the weight."""
    g = gen(11)
    q, cache, table, lens = attention_case([640, 640, 640], 16, 576, 64, seed=11, poison=False)
    flat = cache.view(-1, 576)
    rows = (table.long()[:, :10, None] * 64 + torch.arange(64, device=DEV)).view(3, 640)
    u = randn(g, 576).float()
    ramp = torch.linspace(-3, 3, 640, device=DEV)
    flat[rows[0]] = (ramp[:, None] * u + 0.05 * randn(g, 640, 576).float()).to(torch.bfloat16)
    flat[rows[1]] = flat[rows[0]].flip(0)
    flat[rows[2], :] = (0.01 * randn(g, 640, 576).float()).to(torch.bfloat16)
    flat[rows[2, 333]] = (4 * u).to(torch.bfloat16)
    q[:] = (u[None, None] * torch.linspace(0.1, 1, 16, device=DEV)[None, :, None]).to(torch.bfloat16)
    check_attention(q, cache, table, lens, 512, 0.1)
    check_attention(q, cache, table, lens, 512, 0.002)


def test_attention_bad_pages_read_as_zero_rows_and_are_reported():
    q, cache, table, lens = attention_case([200, 130], 16, 576, 64, seed=12, poison=False)
    clean = cache.clone()
    extra = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device=DEV)
    good = table.clone()
    table[0, 1], table[1, 0] = -1, cache.shape[0]
    good[0, 1] = good[1, 0] = cache.shape[0]
    want = dsnq.paged_latent_attention(q, torch.cat([clean, extra]), good, lens, 512, 0.05)
    assert dsnq.debug_status() == OK
    got = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    assert dsnq.debug_status() == BOUNDS and dsnq.debug_status() == OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    table[0, 1] = 2 ** 31 - 1                                # times the page size it would wrap
    got = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    assert dsnq.debug_status() == BOUNDS and torch.equal(got[0], want[0])


def test_attention_lengths_outside_the_table():
    """A negative length counts as none, one past the table as all of it."""
    q, cache, table, lens = attention_case([192, 100], 8, 576, 64, seed=13, extra=0)
    want = dsnq.paged_latent_attention(q, cache, table, torch.tensor([192, 0], dtype=torch.int32, device=DEV), 512, 0.05)
    got = dsnq.paged_latent_attention(q, cache, table, torch.tensor([5000, -7], dtype=torch.int32, device=DEV), 512, 0.05)
    assert dsnq.debug_status() == OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_strided_views():
    """q, cache, table, out and lse inside wider buffers."""
    lens = [70, 1, 129]
    q, cache, table, n = attention_case(lens, 10, 576, 16, seed=14)
    ref = oracle.paged_latent_attention(val(q), val(cache), table.cpu().numpy(), lens, 512, 0.05)
    wq = torch.full((3, 12, 640), float("nan"), dtype=torch.bfloat16, device=DEV)
    wq[:, 1:11, 64:] = q
    wc = torch.full((cache.shape[0], 20, 592), float("nan"), dtype=torch.bfloat16, device=DEV)
    wc[:, :16, 8:584] = cache
    wt = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wt[:, 1:1 + table.shape[1]] = table
    wo = torch.full((3, 13, 520), 9.0, dtype=torch.bfloat16, device=DEV)
    wl = torch.full((3, 17), 9.0, dtype=torch.float32, device=DEV)
    check_attention(wq[:, 1:11, 64:], wc[:, :16, 8:584], wt[:, 1:1 + table.shape[1]], n, 512, 0.05, ref=ref,
                    out=wo[:, 2:12, :512], lse=wl[:, 3:13])
    assert bool((wo[:, :2] == 9).all()) and bool((wo[:, 12:] == 9).all()) and bool((wo[..., 512:] == 9).all())
    assert bool((wl[:, :3] == 9).all()) and bool((wl[:, 13:] == 9).all())


def test_attention_repeats_and_needs_no_clean_workspace():
    q, cache, table, lens = attention_case([5000, 300, 0, 900], 128, 576, 64, seed=15)
    first = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    ws = torch.full((dsnq.paged_latent_attention_workspace_bytes(4, 128, 512, table.shape[1], 64),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        again = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_a_nan_query_stays_in_its_head():
    q, cache, table, lens = attention_case([200, 90], 20, 576, 64, seed=16)
    want = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    q[0, 3, 7] = float("nan")
    got = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    keep = torch.ones(2, 20, dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    assert bool(torch.isnan(got[0][0, 3]).all())


def test_attention_two_streams_at_once():
    cases = [attention_case([3000, 40, 900], 64, 576, 64, seed=20 + i) for i in range(2)]
    want = [dsnq.paged_latent_attention(*c, 512, 0.05) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = dsnq.paged_latent_attention(*cases[i], 512, 0.05)
    torch.cuda.synchronize()
    assert dsnq.debug_status() == OK
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_attention_on_an_explicit_stream_and_from_threads():
    """A Stream, its handle, and two threads on one stream: the same results."""
    import threading
    cases = [attention_case([2500, 33, 800], 48, 576, 64, seed=80 + i) for i in range(2)]
    want = [dsnq.paged_latent_attention(*c, 512, 0.05) for c in cases]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        got = dsnq.paged_latent_attention(*cases[0], 512, 0.05, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    outs = [[], []]

    def work(i):
        for _ in range(50):
            outs[i].append(dsnq.paged_latent_attention(*cases[i], 512, 0.05))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert len(got) == 50 and all(torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) for g in got)
    assert dsnq.debug_status() == OK


def test_attention_kept_workspace_grows():
    """Small, large and small again on one stream; five streams in turn."""
    for i in range(5):
        with torch.cuda.stream(torch.cuda.Stream()):
            for lens, H in (([3], 16), ([9000, 10], 64), ([70], 16)):
                check_attention(*attention_case(lens, H, 576, 64, seed=90 + i), 512, 0.05)


def test_attention_wait_runs_out_and_is_reported():
    """A copy that never comes: the waits run out, the kernel returns, the
    status is read and cleared, and the next call is right."""
    q, cache, table, lens = attention_case([300, 64], 64, 576, 64, seed=22)
    want = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    torch.cuda.synchronize()
    dsnq.debug_set(1, 20_000_000)
    try:
        dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
        assert dsnq.debug_status() == TIMEOUT
    finally:
        dsnq.debug_set(0, 0)
    assert dsnq.debug_status() == OK
    got = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page", [8, 16])
def test_attention_wait_runs_out_with_many_copies_a_tile(page):
    """Every lane of the copying warp gives up together, whatever it was
    waiting for: long requests in small pages, on every worker."""
    q, cache, table, lens = attention_case([9000, 40, 20000, 0, 700], 80, 576, page, seed=23)
    want = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    torch.cuda.synchronize()
    dsnq.debug_set(1, 5_000_000)
    try:
        for _ in range(3):
            dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
            assert dsnq.debug_status() == TIMEOUT
    finally:
        dsnq.debug_set(0, 0)
    got = dsnq.paged_latent_attention(q, cache, table, lens, 512, 0.05)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and dsnq.debug_status() == OK


# -------------------------------------------------------- a run of them together

class Model:
    """One layer's decode step: 48 heads of 512 columns (wq_b N = 24576), keys
    and values the 512-column latent, the last 64 columns rotated."""

    def __init__(self, B, pages, page, width, rows):
        g = gen(30)
        self.B, self.page, self.rows, self.g = B, page, rows, g
        self.gq, self.gkv = [x.cuda() for x in inputs.gammas(30)]
        self.w1, self.s1 = dsnq.quantize_weight_block128(torch.randn(24576, 1536, generator=g, device=DEV) * 0.02)
        self.w2, self.s2 = dsnq.quantize_weight_block128(torch.randn(256, 1536, generator=g, device=DEV) * 0.02)
        self.f, self.fs = dsnq.rope_frequencies(64, factor=4.0)
        self.cache = torch.full((pages, page, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.scale = 512 ** -0.5

    def step(self, x, lens, new, free):
        """x: the projection rows [rows, 2112] of the step's tokens."""
        q8, qs, kv = dsnq.fused_dual_rmsnorm_group_quant(x[:, :1536], x[:, 1536:2048], self.gq, self.gkv, scale_layout="col")
        qh, _ = dsnq.block_scaled_fp8_gemm_dual(q8, qs, self.w1, self.s1, self.w2, self.s2)
        lens, starts, pos, slots, counts = dsnq.extend_block_tables(lens, new, free, self.table, self.page, x.shape[0])
        dsnq.latent_cache_write(kv, None, pos, slots, self.f, self.cache, rope_scale=self.fs)
        q = dsnq.head_rmsnorm_rope(qh.view(-1, 48, 512), pos, self.f, rope_scale=self.fs)
        return q, kv, lens, starts, pos, slots, counts


def test_decode_step_behind_the_pre_projection():
    """A prompt pass, then three decode steps: every operator's inputs are the
    previous one's outputs; the attention is checked against the oracle on the
    queries and the latents of all steps."""
    B, page = 5, 16
    prompt = [37, 1, 64, 0, 90]
    m = Model(B, 40, page, 8, 0)
    x = randn(m.g, sum(prompt), 2112)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    taken = 0
    _, kv, lens, starts, _, slots, counts = m.step(x, lens, torch.tensor(prompt, dtype=torch.int32, device=DEV), m.free)
    taken += int(counts[0])
    assert lens.tolist() == prompt and int(counts[1]) == int(counts[0]) == sum(-(-n // page) for n in prompt)
    f = m.f.tolist()
    rows = [oracle.latent_rows(val(kv)[starts[b]:starts[b + 1]], None, range(prompt[b]), f, rope_offset=448, rope_scale=m.fs)
            for b in range(B)]
    for step in range(3):
        x = randn(m.g, B, 2112)
        q, kv, lens, _, pos, slots, counts = m.step(x, lens, None, m.free[taken:])
        taken += int(counts[0])
        assert pos.tolist() == [n + step for n in prompt]
        for b in range(B):
            rows[b] = np.concatenate([rows[b], oracle.latent_rows(val(kv)[b:b + 1], None, [prompt[b] + step], f, rope_offset=448,
                                                                  rope_scale=m.fs)])
        got = [val(m.cache.view(-1, 512)[(m.table[b].long()[:, None] * page + torch.arange(page, device=DEV)).view(-1)[:int(lens[b])]])
               for b in range(B)]
        for a, r in zip(got, rows):                          # the cache holds every latent, rounded once
            assert a.shape == r.shape and np.all(np.abs(a - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -14 * 2 * np.abs(r).max())
        check_attention(q, m.cache, m.table, lens, 512, m.scale)
    assert dsnq.debug_status() == OK


def test_decode_step_in_a_graph():
    """The same step captured once and replayed: lengths, tables and cache move
    on on the GPU, and each replay equals the eager step, bit for bit."""
    B, page = 4, 16
    prompt = torch.tensor([15, 0, 31, 60], dtype=torch.int32, device=DEV)

    def build():
        m = Model(B, 40, page, 8, 0)
        x = randn(m.g, int(prompt.sum()), 2112)
        _, _, lens, _, _, _, counts = m.step(x, torch.zeros(B, dtype=torch.int32, device=DEV), prompt, m.free)
        m.lens, m.free = lens, m.free[int(counts[0]):].contiguous()
        m.x = torch.zeros(B, 2112, dtype=torch.bfloat16, device=DEV)
        m.ws = torch.empty(dsnq.paged_latent_attention_workspace_bytes(B, 48, 512, 8, page), dtype=torch.uint8, device=DEV)
        return m

    def step(m):
        q, _, lens, _, _, _, counts = m.step(m.x, m.lens, None, m.free)
        out, lse = dsnq.paged_latent_attention(q, m.cache, m.table, lens, 512, m.scale, workspace=m.ws)
        m.lens.copy_(lens)
        idx = (torch.arange(m.free.numel(), device=DEV) + counts[0]) % m.free.numel()
        m.free.copy_(m.free[idx])
        return out, lse

    eager, cap = build(), build()
    s = torch.cuda.Stream()
    saved = [t.clone() for t in (cap.lens, cap.free, cap.table, cap.cache)]
    with torch.cuda.stream(s):
        step(cap)                                            # warm up, then put the state back
        torch.cuda.synchronize()
        for t, v in zip((cap.lens, cap.free, cap.table, cap.cache), saved):
            t.copy_(v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, lse = step(cap)
    torch.cuda.synchronize()
    for i in range(5):
        x = randn(gen(40 + i), B, 2112)
        eager.x.copy_(x)
        cap.x.copy_(x)
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(cap.lens, eager.lens) and torch.equal(cap.table, eager.table)
    assert dsnq.debug_status() == OK


def test_launch_overlap_changes_nothing():
    q, cache, table, lens = attention_case([900, 64, 0], 48, 576, 64, seed=41)
    pos = torch.arange(3, device=DEV)

    def chain():
        x = dsnq.head_rmsnorm_rope(q, pos, FREQ(64))
        return [x, *dsnq.paged_latent_attention(x, cache, table, lens, 512, 0.05)]

    on = chain()
    dsnq.set_launch_overlap(False)
    try:
        off = chain()
    finally:
        dsnq.set_launch_overlap(True)
    assert all(torch.equal(a, b) for a, b in zip(on, off))


_FIRST_CALLS_IN_CAPTURE = """
import torch
import gemm_dsnq_dual_gb300 as dsnq
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
f, _ = dsnq.rope_frequencies(64)
kv, q = torch.randn(3, 512, device="cuda").bfloat16(), torch.randn(2, 48, 512, device="cuda").bfloat16()
cache = torch.zeros(8, 64, 512, dtype=torch.bfloat16, device="cuda")

def step():
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    lens, _, pos, slots, _ = dsnq.extend_block_tables(lens0, new, free, table, 64, 3)
    dsnq.latent_cache_write(kv, None, pos, slots, f, cache)
    qr = dsnq.head_rmsnorm_rope(q, pos[:2], f)
    return dsnq.paged_latent_attention(qr, cache, table, lens, 512, 0.05)

lens0, new, free = i32([0, 0]), i32([2, 1]), i32([5, 6])
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    out = step()
g.replay()
torch.cuda.synchronize()
want = step()
assert dsnq.debug_status() == 0
assert all(torch.equal(a, b) for a, b in zip(out, want)) and bool(out[0].isfinite().all()) and bool((out[0] != 0).any())
print("captured ok")
"""


def test_first_calls_may_be_captured():
    """In a fresh process: each operator's first call is made under capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr


def test_two_graphs_at_once():
    """Two captured calls, replayed at the same time on two streams: each has
    its own workspace from its graph's pool."""
    cases = [attention_case([4000, 77, 900], 64, 576, 64, seed=70 + i) for i in range(2)]
    want = [dsnq.paged_latent_attention(*c, 512, 0.05) for c in cases]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(dsnq.paged_latent_attention(*c, 512, 0.05))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_empty_calls():
    e = torch.empty(0, 512, dtype=torch.bfloat16, device=DEV)
    i = torch.empty(0, dtype=torch.int64, device=DEV)
    cache = torch.ones(2, 8, 512, dtype=torch.bfloat16, device=DEV)
    dsnq.latent_cache_write(e, None, i, i, FREQ(64), cache)
    assert bool((cache == 1).all()) and dsnq.debug_status() == OK


def test_other_device_is_refused():
    """Tensors that are not on the current device are refused by name."""
    cpu = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsnq.head_rmsnorm_rope(cpu, torch.zeros(1, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))


def test_debug_build_checks_every_index():
    """The debug build's index checks pass on small cases of each kernel, with
    the release build's results."""
    from gemm_dsnq_dual_gb300 import _native
    release = _native.LIB_PATH

    def run():
        outs = []
        for layout in ("interleaved", "half"):
            for D in (64, 128, 192, 512, 576):
                outs.append(dsnq.head_rmsnorm_rope(randn(gen(50), 3, 5, D), torch.arange(3, device=DEV), FREQ(64), layout=layout))
            for K, P in ((192, 0), (256, 64), (512, 64), (768, 64)):
                cache = torch.zeros(4, 8, K + P, dtype=torch.bfloat16, device=DEV)
                pe = randn(gen(51), 9, P) if P else None
                dsnq.latent_cache_write(randn(gen(52), 9, K), pe, torch.arange(9, device=DEV), torch.arange(9, device=DEV) * 3, FREQ(64),
                                        cache, normalize=True, layout=layout)
                outs.append(cache)
        lens, new, free, table, _ = extend_case(40, 8, seed=53)
        t = torch.tensor(table, dtype=torch.int32, device=DEV)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        outs += [*dsnq.extend_block_tables(i32(lens), i32(new), i32(free), t, 8, int(new.sum())), t]
        for H, lens in ((16, [700, 0, 65]), (100, [300, 5]), (48, [64] * 200)):
            outs += dsnq.paged_latent_attention(*attention_case(lens, H, 576, 16, seed=54), 512, 0.05)
        torch.cuda.synchronize()
        return outs

    want = run()
    try:
        _native.use_library(_native.DEBUG_LIB_PATH)
        got = run()
        assert dsnq.debug_status() == OK
    finally:
        _native.use_library(release)
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(got, want))
