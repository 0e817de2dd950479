"""The decode-step operators without a GPU: pins of their oracle against
formulas written another way, and the argument checks of the C ABI and the
binding (nothing here reaches the CUDA runtime)."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq
import oracle
from gemm_dsnq_dual_gb300 import _native, build
from gemm_dsnq_dual_gb300.inputs import bits

OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.lib()


# ------------------------------------------------------------- oracle pins

def test_decode_bf16_agrees_with_torch():
    x = torch.randn(1000).to(torch.bfloat16)
    assert np.array_equal(oracle.decode_bf16(bits(x)), x.double().numpy())


def test_extend_hand_case():
    """Three requests, pages of 4: 5 tokens + 1 (fits its second page), 4 + 2
    (opens one), none + 5 (opens two)."""
    table = [[7, 3, -1], [5, -1, -1], [-1, -1, -1]]
    lens, starts, pos, slots, counts, t = oracle.extend_block_tables([5, 4, 0], [1, 2, 5], [9, 8, 2, 6], table, 4, 10)
    assert lens.tolist() == [6, 6, 5] and starts.tolist() == [0, 1, 3, 8] and counts.tolist() == [3, 3]
    assert pos.tolist() == [5, 4, 5, 0, 1, 2, 3, 4, 0, 0]
    assert slots.tolist() == [13, 36, 37, 32, 33, 34, 35, 8, -1, -1]
    assert t.tolist() == [[7, 3, -1], [5, 9, -1], [8, 2, -1]]
    # One free page: the second request takes it, the third gets no place.
    lens, _, _, slots, counts, _ = oracle.extend_block_tables([5, 4, 0], [1, 2, 5], [9], table, 4, 10)
    assert lens.tolist() == [6, 6, 0] and counts.tolist() == [1, 3] and slots.tolist() == [13, 36, 37] + [-1] * 7


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 8)), [0, 1, 17, 4095, 1 << 20]
    f = 10000.0 ** (-np.arange(4) / 4)
    z = np.exp(1j * np.outer(pos, f))[:, None]
    y = oracle.rope_rotate(x, pos, f, "interleaved", 1.5)
    w = (x[..., 0::2] + 1j * x[..., 1::2]) * z * 1.5
    assert np.allclose(y[..., 0::2], w.real, atol=1e-9) and np.allclose(y[..., 1::2], w.imag, atol=1e-9)
    h = oracle.rope_rotate(x, pos, f, "half")
    w = (x[..., :4] + 1j * x[..., 4:]) * z
    assert np.allclose(h[..., :4], w.real, atol=1e-9) and np.allclose(h[..., 4:], w.imag, atol=1e-9)
    assert np.allclose(oracle.rope_rotate(h, pos, f, "half", inverse=True), x, atol=1e-9)


def test_rotation_at_far_positions_is_exact():
    """The angle is the exact product's: at 2^50 an fp64 product is off by up
    to 2^-4 rad, the exact fraction of a turn, rounded once to fp64, by 2^-51."""
    from fractions import Fraction
    per_turn = Fraction("0.159154943091895335768883763372514362034459645740456448747667344")   # 1 / (2 pi)
    pos, f = [2**50 + 1, -(2**50) - 12345, 2**62 - 1, 2**31 - 1, 3], [0.1, 1.0, 1e-5, 0.7320508]
    x = np.zeros((len(pos), 8))
    x[:, 0::2] = 1
    y = oracle.rope_rotate(x, pos, f, "interleaved")
    for i, p in enumerate(pos):
        for j, w in enumerate(f):
            t = float((p * Fraction(w) * per_turn) % 1) * 2 * math.pi
            assert abs(y[i, 2 * j] - math.cos(t)) < 1e-14 and abs(y[i, 2 * j + 1] - math.sin(t)) < 1e-14


def test_norm_agrees_with_torch():
    x, g = torch.randn(4, 3, 32, dtype=torch.float64), torch.rand(32, dtype=torch.float64)
    y = oracle.head_rmsnorm_rope(x.numpy(), [0] * 4, [], g.numpy(), 1e-5)
    assert np.allclose(y, torch.nn.functional.rms_norm(x, (32,), g, 1e-5).numpy(), rtol=1e-12)
    rows = oracle.latent_rows(x[:, 0].numpy(), x[:, 1, :8].numpy(), [0] * 4, [], g.numpy(), 1e-5, True)
    assert np.allclose(rows[:, :32], y[:, 0]) and np.array_equal(rows[:, 32:], x[:, 1, :8].numpy())


def test_attention_agrees_with_a_dense_softmax():
    rng = np.random.default_rng(1)
    cache, q = rng.standard_normal((5, 4, 16)), rng.standard_normal((3, 2, 16))
    table, lens = [[3, 0, 1], [2, -1, -1], [4, -1, -1]], [9, 0, 1]
    out, lse, _, _ = oracle.paged_latent_attention(q, cache, table, lens, 8, 0.3)
    k = torch.tensor(cache[[3, 0, 1]].reshape(-1, 16)[:9])
    z = torch.tensor(q[0]) @ k.T * 0.3
    assert np.allclose(out[0], (z.softmax(-1) @ k[:, :8]).numpy()) and np.allclose(lse[0], z.logsumexp(-1).numpy())
    assert np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
    assert np.allclose(out[2], cache[4, 0, :8])          # one token: its value


# --------------------------------------------------------- rotary frequencies

def test_rope_frequencies():
    f, s = dsnq.rope_frequencies(64, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    g, s = dsnq.rope_frequencies(64, factor=16.0, original_length=4096, device="cpu")
    assert math.isclose(s, 0.1 * math.log(16) + 1)
    turns = f * 4096 / (2 * math.pi)
    r = g / f
    assert torch.all(r[turns > 40] == 1.0) and torch.allclose(r[turns < 0.8], torch.tensor(1 / 16, dtype=torch.float64))
    assert torch.all(r[1:] <= r[:-1] + 1e-15)             # one ramp between
    with pytest.raises(ValueError):
        dsnq.rope_frequencies(7, device="cpu")


# -------------------------------------------------------------- C ABI refusals

def test_extend_argument_checks(lib):
    def call(B=4, rows=8, ps=16, lens=A, new=A + 64, free=A, F=10, table=A, width=8, ld=8, nl=A + 256, rs=A + 512, pos=A,
             slots=A + 1024, counts=A):
        return lib.dsnq_extend_block_tables(B, rows, ps, lens, new, free, F, table, width, ld, nl, rs, pos, slots, counts, None)

    assert call(B=-1) == INVALID and call(rows=-1) == INVALID and call(ps=0) == INVALID and call(F=-1) == INVALID
    assert call(width=-1) == INVALID
    assert call(B=8193) == UNSUPPORTED                       # DSNQ_MAX_REQUESTS
    assert call(ps=1 << 21) == UNSUPPORTED
    assert call(width=1 << 20, ld=1 << 20, ps=1 << 12) == UNSUPPORTED      # tokens of a request beyond int32
    assert call(width=1 << 62, ld=1 << 62) == UNSUPPORTED
    assert call(rows=1 << 31) == UNSUPPORTED
    for name in ("lens", "table", "nl", "rs", "pos", "slots", "counts", "free"):
        assert call(**{name: None}) == INVALID, name
    assert call(ld=7) == INVALID
    assert call(nl=A) == INVALID                              # the lengths in place
    assert call(rs=A) == INVALID
    assert call(nl=A + 64) == INVALID                         # the counts in place
    assert call(slots=A) == INVALID and call(rs=A + 256) == INVALID        # two outputs in one place
    assert call(lens=A + 2) == MISALIGNED and call(slots=A + 4) == MISALIGNED and call(pos=A + 4) == MISALIGNED


def test_head_norm_rope_argument_checks(lib):
    def call(M=4, H=3, D=64, x=A, lt=192, lh=64, norm=1, gamma=None, eps=1e-6, pos=A, f=A, off=0, dim=64, lay=0, scale=1.0,
             inv=0, out=2 * A, ot=192, oh=64):
        return lib.dsnq_head_rmsnorm_rope(M, H, D, x, lt, lh, norm, gamma, eps, pos, f, off, dim, lay, scale, inv, out, ot, oh, None)

    assert call(M=0) == OK and call(M=0, x=None, out=None, pos=None, f=None) == OK
    assert call(M=-1) == INVALID and call(H=0) == INVALID and call(D=0) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(norm=0, gamma=A) == INVALID                   # a weight without a norm
    assert call(D=60) == UNSUPPORTED and call(D=1032, lh=1032, lt=3 * 1032, oh=1032, ot=3 * 1032) == UNSUPPORTED
    assert call(H=65536) == UNSUPPORTED
    assert call(off=8) == INVALID and call(off=-8) == INVALID and call(dim=-16) == INVALID     # outside the head
    assert call(off=1 << 62) == INVALID
    assert call(dim=40) == UNSUPPORTED and call(off=4, dim=32) == UNSUPPORTED
    assert call(D=512, lh=512, lt=1536, oh=512, ot=1536, dim=512) == UNSUPPORTED               # more than 256 columns
    assert call(lay=2) == INVALID and call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    assert call(x=None) == INVALID and call(out=None) == INVALID and call(pos=None) == INVALID and call(f=None) == INVALID
    assert call(lh=56) == INVALID and call(ot=56) == INVALID
    assert call(out=A, ot=256) == INVALID and call(out=A, oh=128, ot=384) == INVALID           # in place, other strides
    assert call(x=A + 8) == MISALIGNED and call(lt=196) == MISALIGNED and call(gamma=A + 2) == MISALIGNED
    assert call(pos=A + 4) == MISALIGNED and call(f=A + 4) == MISALIGNED


def test_cache_write_argument_checks(lib):
    def call(M=4, K=512, P=64, kv=A, ldkv=2112, pe=A, ldpe=2112, norm=0, gamma=None, eps=1e-6, pos=A, f=A, off=512, dim=64,
             lay=0, scale=1.0, slots=A, cache=A, pages=4, ps=16, lp=16 * 576, lr=576):
        return lib.dsnq_latent_cache_write(M, K, P, kv, ldkv, pe, ldpe, norm, gamma, eps, pos, f, off, dim, lay, scale, slots,
                                           cache, pages, ps, lp, lr, None)

    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(K=0) == INVALID and call(P=-8) == INVALID and call(pages=-1) == INVALID
    assert call(ps=0) == INVALID
    assert call(K=500) == UNSUPPORTED and call(P=60) == UNSUPPORTED and call(K=1024, lr=1088, lp=16 * 1088) == UNSUPPORTED
    assert call(ps=1 << 21, lp=1 << 40) == UNSUPPORTED
    assert call(kv=None) == INVALID and call(pe=None) == INVALID and call(slots=None) == INVALID and call(cache=None) == INVALID
    assert call(gamma=A) == INVALID                           # a weight without a norm
    assert call(norm=1, eps=float("nan")) == INVALID
    assert call(off=520) == INVALID and call(off=516, dim=32) == UNSUPPORTED
    assert call(ldkv=500) == INVALID and call(lr=568) == INVALID and call(lp=16 * 576 - 8) == INVALID
    assert call(kv=A + 8) == MISALIGNED and call(lr=580, lp=16 * 580) == MISALIGNED and call(cache=A + 2) == MISALIGNED
    assert call(slots=A + 4) == MISALIGNED


def test_attention_argument_checks(lib):
    n = C.c_int64()
    assert lib.dsnq_paged_latent_attention_workspace_bytes(4, 128, 512, 16, 64, C.byref(n)) == OK
    ws = n.value

    def call(B=4, H=128, DK=576, DV=512, q=A, qt=128 * 576, qh=576, cache=A, pages=9, ps=64, lp=64 * 576, lr=576, table=A,
             width=16, ldt=16, lens=A, scale=0.1, out=A, ot=128 * 512, oh=512, lse=A, ll=128, w=A, wb=ws):
        return lib.dsnq_paged_latent_attention(B, H, DK, DV, q, qt, qh, cache, pages, ps, lp, lr, table, width, ldt, lens, scale,
                                               out, ot, oh, lse, ll, w, wb, None)

    assert call(B=0) == OK
    assert call(B=-1) == INVALID and call(H=0) == INVALID and call(width=-1) == INVALID and call(ps=0) == INVALID
    assert call(pages=0) == INVALID
    assert call(DV=640) == INVALID                            # a value wider than the row
    assert call(DK=560) == UNSUPPORTED and call(DK=640, qh=640, qt=128 * 640, lr=640, lp=64 * 640) == UNSUPPORTED
    assert call(DV=448) == UNSUPPORTED and call(H=1025) == UNSUPPORTED and call(B=8193) == UNSUPPORTED
    assert call(ps=60) == UNSUPPORTED and call(ps=4) == UNSUPPORTED
    assert call(lr=1 << 20, lp=1 << 21) == INVALID            # pages that overlap
    assert call(ps=8, lr=1 << 36, lp=1 << 39, width=1, ldt=1) == UNSUPPORTED and call(qt=1 << 39) == UNSUPPORTED
    assert call(width=1 << 26, ldt=1 << 26) == UNSUPPORTED    # tokens of a request beyond int32
    assert call(scale=0.0) == INVALID and call(scale=-1.0) == INVALID and call(scale=float("nan")) == INVALID
    for name in ("q", "cache", "table", "lens", "out", "w"):
        assert call(**{name: None}) == INVALID, name
    assert call(qh=568) == INVALID and call(ot=504) == INVALID and call(ldt=15) == INVALID and call(ll=127) == INVALID
    assert call(lr=568) == INVALID and call(lp=64 * 576 - 8) == INVALID
    assert call(wb=ws - ws // 2) == INVALID                   # workspace too small
    assert call(q=A + 8) == MISALIGNED and call(lr=580, lp=64 * 580) == MISALIGNED and call(w=A + 8) == MISALIGNED
    assert call(lens=A + 2) == MISALIGNED


def test_attention_workspace_query(lib):
    """Grows with the workers a call can have, up to the whole GPU's."""
    def size(B, H, DV=512, width=16, ps=64):
        return dsnq.paged_latent_attention_workspace_bytes(B, H, DV, width, ps)

    assert size(0, 128) == 0
    assert size(1, 128, width=1) < size(1, 128) <= size(64, 128) == size(1000, 128)
    assert size(1000, 128) < 43 << 20 and size(8192, 16, width=1000) < 43 << 20
    n = C.c_int64()
    q = lib.dsnq_paged_latent_attention_workspace_bytes
    assert q(4, 128, 500, 16, 64, C.byref(n)) == UNSUPPORTED and q(-1, 128, 512, 16, 64, None) == INVALID
    assert q(1 << 40, 128, 512, 16, 64, None) == UNSUPPORTED


# ------------------------------------------------------------ binding refusals

def test_binding_refuses_wrong_types_and_shapes():
    """Checked before the library is called (the tensors are on the CPU)."""
    i32, i64, bf = torch.int32, torch.int64, torch.bfloat16
    x = torch.zeros(4, 3, 64, dtype=bf)
    pos, f = torch.zeros(4, dtype=i64), torch.zeros(32, dtype=torch.float64)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(positions=pos.int()), dict(positions=pos[:3]), dict(inv_freq=f.float()),
                dict(out=torch.zeros(4, 3, 32, dtype=bf)), dict(gamma=torch.zeros(32, dtype=bf)), dict(layout="other"),
                dict(x=torch.zeros(4, 64, 3, dtype=bf).transpose(1, 2))):
        a = dict(x=x, positions=pos, inv_freq=f)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsnq.head_rmsnorm_rope(**a)
    kv, pe, cache = torch.zeros(4, 512, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(2, 16, 576, dtype=bf)
    for bad in (dict(kv=kv.float()), dict(pe=pe[:3]), dict(slots=pos.int()), dict(cache=cache[..., :512]), dict(pe=None)):
        a = dict(kv=kv, pe=pe, positions=pos, slots=pos, inv_freq=f, cache=cache)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsnq.latent_cache_write(**a)
    q, table, lens = torch.zeros(4, 8, 576, dtype=bf), torch.zeros(4, 2, dtype=i32), torch.zeros(4, dtype=i32)
    for bad in (dict(q=q[..., :512]), dict(block_table=table.long()), dict(block_table=table[:3]), dict(seq_lens=lens.long()),
                dict(out=torch.zeros(4, 8, 576, dtype=bf)), dict(lse=torch.zeros(4, 8)[:, :4]),
                dict(workspace=torch.zeros(8, dtype=torch.float32))):
        a = dict(q=q, cache=cache, block_table=table, seq_lens=lens, v_dim=512, scale=0.1)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsnq.paged_latent_attention(**a)
    for bad in (dict(seq_lens=lens.long()), dict(new_tokens=lens[:2]), dict(block_table=table.t())):
        a = dict(seq_lens=lens, new_tokens=lens, free_pages=lens, block_table=table, page_size=16, rows=4)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dsnq.extend_block_tables(**a)
