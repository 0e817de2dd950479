"""The debug build (libdsnq_debug.so, compiled with DSNQ_DEBUG): every
kernel checks the indices of its memory accesses against the extents its
arguments describe.  One small case per kernel runs under it, its results are
checked against the release build bit for bit, and the device status words
must report no failed check; the reporting path itself is exercised with the
hook that records one deliberate failed check guarding no access."""

import numpy as np
import pytest
import torch

import oracle
import gemm_dsnq_dual_gb300 as dsnq
from gemm_dsnq_dual_gb300 import _native, inputs

pytestmark = pytest.mark.gpu
OK, BOUNDS = 0, 6


@pytest.fixture(scope="module")
def libs():
    release = _native.LIB_PATH
    yield release, _native.DEBUG_LIB_PATH
    _native.use_library(release)


def run_every_kernel():
    """One small call of each kernel; returns every output tensor."""
    outs = []
    lat = inputs.decode_batch(4, seed=31)                     # warp-group-per-row kernel, split views
    buf = lat.buf.cuda()
    gq, gkv = lat.gamma_q.cuda(), lat.gamma_kv.cuda()
    outs += dsnq.fused_dual_rmsnorm_group_quant(buf[:, :1536], buf[:, 1536:2048], gq, gkv, lat.eps, scale_layout="col")
    big = inputs.full_path_batch(1536, seed=32)               # DSv4 warp-per-row kernel (M >= 8 x SMs)
    q, kv = big.q.cuda(), big.kv.cuda()
    outs += dsnq.fused_dual_rmsnorm_group_quant(q, kv, gq, gkv, lat.eps, scale_layout="row")
    outs += dsnq.rmsnorm_group_quant(q[:5], gq, lat.eps)      # single latent
    qb, kvb = dsnq.dual_rmsnorm_bf16(q, kv, gq, gkv, lat.eps)  # unfused baseline, warp-per-row modes
    outs += [qb, kvb]
    outs += dsnq.group_quant_bf16(qb, scale_layout="col")
    outs += dsnq.group_quant_bf16(qb[:7])                     # warp-group mode
    outs += dsnq.quantize_weight_block128(inputs.weight(300, 1536, seed=33).cuda())
    w1, s1 = dsnq.quantize_weight_block128(inputs.weight(512, 1536, seed=34).cuda())
    w2, s2 = dsnq.quantize_weight_block128(inputs.weight(256, 1536, seed=35).cuda())
    for M in (3, 40, 100, 300):                               # decode, decode BN=64, 128x128 tiles, CTA pair
        a8, sa = dsnq.fused_dual_rmsnorm_group_quant(q[:M], kv[:M], gq, gkv, lat.eps, scale_layout="col")[:2]
        outs += dsnq.block_scaled_fp8_gemm_dual(a8, sa, w1, s1, w2, s2)
    xa = inputs.activations_bf16(2, 1536, seed=36).cuda()
    outs += dsnq.block_scaled_fp8_gemm_dual_bf16a(xa, w1, s1, w2, s2)         # quantized in the prologue
    outs += dsnq.fused_norm_quant_gemm_dual(buf[:2, :1536], buf[:2, 1536:2048], gq, gkv, lat.eps, w1, s1, w2, s2)[:3]
    torch.cuda.synchronize()
    return outs


def as_bits(t):
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        return t.contiguous().view(torch.uint8)
    return t.contiguous().view(torch.int16) if t.element_size() == 2 else t.contiguous().view(torch.int32)


def test_every_kernel_passes_its_index_checks_and_matches_the_release_build(libs):
    release, debug = libs
    _native.use_library(release)
    want = run_every_kernel()
    _native.use_library(debug)
    assert _native.lib().dsnq_debug_build() == 1
    assert dsnq.debug_status() == OK
    got = run_every_kernel()
    assert dsnq.debug_status() == OK                          # no check failed
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert torch.equal(as_bits(g), as_bits(w))


def test_a_failed_check_is_reported_and_cleared(libs):
    """The hook records one failed check per launch without any access
    attached; dsnq_debug_status reports it once and clears the words."""
    _, debug = libs
    _native.use_library(debug)
    lat = inputs.pr1_ref(0)
    args = (lat.q.cuda(), lat.kv.cuda(), lat.gamma_q.cuda(), lat.gamma_kv.cuda(), lat.eps)
    ref = dsnq.fused_dual_rmsnorm_group_quant(*args)
    assert dsnq.debug_status() == OK
    dsnq.debug_set(inject_flags=2)
    try:
        got = dsnq.fused_dual_rmsnorm_group_quant(*args)
        assert dsnq.debug_status() == BOUNDS
    finally:
        dsnq.debug_set(0, 0)
    assert dsnq.debug_status() == OK
    for g, w in zip(got, ref):                                # the computation itself is unaffected
        assert torch.equal(as_bits(g), as_bits(w))
    codes, scale, _ = oracle.fused_dual_rmsnorm_group_quant(*[inputs.bits(t) for t in
                                                             (lat.q, lat.kv, lat.gamma_q, lat.gamma_kv)], lat.eps)
    assert np.array_equal(scale, got[1].cpu().numpy()) or np.allclose(scale, got[1].cpu().numpy(), rtol=1e-6)


@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("H", [16, 32, 48, 64])
def test_sums_of_a_job_outlive_their_late_readers(libs, H, prefix):
    """Attention over an 8-bit cache, several requests a worker: the warps of a
    job read one another's sums at its end.  The hook lets a quarter of them
    come late to that; the others may not have written over the sums by then."""
    _, debug = libs
    _native.use_library(debug)
    g = torch.Generator(device="cuda")
    g.manual_seed(H + prefix)
    B, page, K = 400, 64, 256
    lens = torch.randint(1, 300, (B,), generator=g, device="cuda").to(torch.int32)
    pages = 40
    cache = (torch.randn(pages, page, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.rand(pages, page, generator=g, device="cuda") * 0.01
    table = torch.randint(0, pages, (B, 5), generator=g, device="cuda").to(torch.int32)
    q = torch.randn(B, H, K, generator=g, device="cuda").to(torch.bfloat16)
    front, front_len = torch.arange(5, dtype=torch.int32, device="cuda"), torch.tensor([prefix], dtype=torch.int32, device="cuda")

    def call():
        if prefix:
            return dsnq.shared_prefix_latent_attention_fp8(q, cache, scales, front, front_len, table, lens, K, 0.1)
        return dsnq.paged_latent_attention_fp8(q, cache, scales, table, lens, K, 0.1)

    want = call()
    assert dsnq.debug_status() == OK
    dsnq.debug_set(inject_flags=4)
    try:
        got = call()
        assert dsnq.debug_status() == OK
    finally:
        dsnq.debug_set(0, 0)
    for a, b in zip(got, want):
        assert torch.equal(as_bits(a), as_bits(b))


def run_decode_step_kernels():
    """One small call of each kernel of the decode step's other operators;
    returns every output tensor."""
    outs = []
    g = torch.Generator(device="cuda")
    g.manual_seed(41)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    B, page, prefix = 9, 16, 200
    freq, _ = dsnq.rope_frequencies(64, device="cuda")
    for layout in ("interleaved", "half"):
        outs.append(dsnq.head_rmsnorm_rope(randn(7, 5, 192), torch.arange(7, device="cuda") * 1000, freq, layout=layout))
    # Requests of up to 1700 tokens and an empty one, before one more token each; odd pages, a table with room.
    lens = ints([1699, 1, 127, 128, 300, 0, 40, 900, 15])
    held = [-(-n // page) for n in lens.tolist()]
    pages = sum(held) + B + 16
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((B, 120), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    front, free = ids[at:at + 13].clone(), ids[at + 13:].clone()
    lens, starts, positions, slots, counts = dsnq.extend_block_tables(lens, None, free, table, page, B + 3)
    outs += [lens, starts, positions, slots, counts, table]
    kv, pe = randn(B + 3, 512), randn(B + 3, 64)
    wide = randn(pages, page, 576)
    codes = torch.cat([(wide[..., :512].float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8),
                       (wide[..., 512:].float() * 100).to(torch.bfloat16).view(torch.uint8)], -1)
    scales = torch.rand(pages, page, generator=g, device="cuda") * 0.02
    for layout in ("interleaved", "half"):
        dsnq.latent_cache_write(kv, pe, positions, slots, freq, wide, normalize=True, layout=layout)
        dsnq.latent_cache_write_fp8(kv, pe, positions, slots, freq, codes, scales, normalize=True, layout=layout)
        outs += [wide.clone(), codes.clone(), scales.clone()]
    total = int(lens.sum())
    reads = torch.cat([ints([0]), lens.cumsum(0).to(torch.int32)])
    outs.append(dsnq.latent_cache_read_fp8(codes, scales, 512, table, reads, total))                    # short: 8 rows a CTA
    many = 5 * total
    row_starts = torch.cat([ints([0])] + [reads[1:] + i * total for i in range(5)])
    outs.append(dsnq.latent_cache_read_fp8(codes, scales, 512, table.repeat(5, 1), row_starts, many))   # 16 rows a CTA
    # Attention: every count of heads that has a kernel, with and without position columns and a prefix, tables with
    # and without room (CTAs of 16, 32 and 64 heads), many requests (several a worker).
    narrow = codes[..., :512]
    room = torch.cat([table, torch.full((B, 30000), -1, dtype=torch.int32, device="cuda")], 1)
    for H in (7, 16, 32, 48, 64, 130):
        q = randn(B, H, 576)
        outs += dsnq.paged_latent_attention(q, wide, table, lens, 512, 0.05)
        for t in (table, room):
            outs += dsnq.paged_latent_attention_fp8(q, codes, scales, t, lens, 512, 0.05)
            outs += dsnq.shared_prefix_latent_attention_fp8(q, codes, scales, front, ints([prefix]), t, lens, 512, 0.05)
        outs += dsnq.paged_latent_attention_fp8(q[..., :512], narrow, scales, table, lens, 256, 0.05)
        rows = torch.arange(400, device="cuda") % B
        outs += dsnq.paged_latent_attention_fp8(q[rows], codes, scales, table[rows], lens[rows], 512, 0.05)
        outs += dsnq.shared_prefix_latent_attention_fp8(q[rows], codes, scales, front, ints([prefix]), table[rows], lens[rows], 512, 0.05)
    torch.cuda.synchronize()
    return outs


def test_decode_step_kernels_pass_their_index_checks_and_match_the_release_build(libs):
    release, debug = libs
    _native.use_library(release)
    want = run_decode_step_kernels()
    _native.use_library(debug)
    assert dsnq.debug_status() == OK
    got = run_decode_step_kernels()
    assert dsnq.debug_status() == OK                          # no check failed
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert g.dtype == w.dtype and torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))
