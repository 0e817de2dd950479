"""The latent cache in 8 bits without a GPU: the argument checks of the C ABI
(nothing here reaches the CUDA runtime), and the binding against a recording
library: what it hands on, and that each wrong argument is refused by name."""

import ctypes as C

import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq
from gemm_dsnq_dual_gb300 import _native, build

OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
I32, I64, BF, F32, F64, U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.float64, torch.uint8


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.lib()


# ---------------------------------------------------------------- C ABI checks

def test_write_argument_checks(lib):
    def call(M=4, K=512, P=64, kv=A, ldkv=2112, pe=A, ldpe=2112, norm=0, gamma=None, eps=1e-6, pos=A, f=A, off=512, dim=64,
             lay=0, scale=1.0, slots=A, cache=A, pages=4, ps=16, lp=16 * 640, lr=640, scales=A, lds=16):
        return lib.dsnq_latent_cache_write_fp8(M, K, P, kv, ldkv, pe, ldpe, norm, gamma, eps, pos, f, off, dim, lay, scale, slots,
                                               cache, pages, ps, lp, lr, scales, lds, None)

    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(K=0) == INVALID and call(P=-8) == INVALID and call(pages=-1) == INVALID and call(ps=0) == INVALID
    assert call(K=500) == UNSUPPORTED and call(P=60) == UNSUPPORTED and call(K=1024, lr=1152, lp=16 * 1152) == UNSUPPORTED
    assert call(K=504, off=504) == UNSUPPORTED and call(M=0, K=504, off=504) == UNSUPPORTED      # position columns off their 16 bytes
    assert call(ps=1 << 21, lp=1 << 40) == UNSUPPORTED
    for name in ("kv", "pe", "slots", "cache", "scales"):
        assert call(**{name: None}) == INVALID, name
    assert call(gamma=A) == INVALID and call(norm=1, eps=float("nan")) == INVALID
    assert call(off=520) == INVALID and call(off=516, dim=32) == UNSUPPORTED
    assert call(ldkv=500) == INVALID and call(lr=624) == INVALID and call(lp=16 * 640 - 16) == INVALID and call(lds=15) == INVALID
    assert call(kv=A + 8) == MISALIGNED and call(lr=648, lp=16 * 648) == MISALIGNED and call(cache=A + 8) == MISALIGNED
    assert call(slots=A + 4) == MISALIGNED and call(scales=A + 2) == MISALIGNED


def test_read_argument_checks(lib):
    def call(B=4, rows=9, K=512, P=64, cache=A, pages=4, ps=16, lp=16 * 640, lr=640, scales=A, lds=16, table=A, width=3, ldt=3,
             starts=A, first=A, out=A, ldo=576):
        return lib.dsnq_latent_cache_read_fp8(B, rows, K, P, cache, pages, ps, lp, lr, scales, lds, table, width, ldt, starts, first,
                                              out, ldo, None)

    assert call(B=0) == OK and call(rows=0) == OK
    assert call(B=-1) == INVALID and call(rows=-1) == INVALID and call(K=0) == INVALID and call(P=-8) == INVALID
    assert call(pages=-1) == INVALID and call(ps=0) == INVALID and call(width=-1) == INVALID
    assert call(K=504) == UNSUPPORTED and call(P=4) == UNSUPPORTED and call(K=1024) == UNSUPPORTED and call(B=8193) == UNSUPPORTED
    assert call(width=1 << 28, ldt=1 << 28) == UNSUPPORTED and call(ps=1 << 21) == UNSUPPORTED and call(rows=1 << 31) == UNSUPPORTED
    for name in ("cache", "scales", "table", "starts", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(ldo=568) == INVALID and call(ldt=2) == INVALID and call(lr=624) == INVALID and call(lp=16 * 640 - 16) == INVALID
    assert call(lds=15) == INVALID
    assert call(cache=A + 8) == MISALIGNED and call(lr=648, lp=16 * 648) == MISALIGNED and call(out=A + 8) == MISALIGNED
    assert call(ldo=580) == MISALIGNED and call(starts=A + 2) == MISALIGNED and call(first=A + 1) == MISALIGNED


@pytest.mark.parametrize("shared", [False, True])
def test_attention_argument_checks(lib, shared):
    n = C.c_int64()
    if shared:
        assert lib.dsnq_shared_prefix_latent_attention_fp8_workspace_bytes(4, 128, 512, 20, 16, 64, C.byref(n)) == OK
    else:
        assert lib.dsnq_paged_latent_attention_fp8_workspace_bytes(4, 128, 512, 16, 64, C.byref(n)) == OK
    ws = n.value

    def call(B=4, H=128, K=512, P=64, DV=512, q=A, qt=128 * 576, qh=576, cache=A, pages=9, ps=64, lp=64 * 640, lr=640, scales=A,
             lds=64, ptable=A, pwidth=20, plen=A, table=A, width=16, ldt=16, lens=A, scale=0.1, out=A, ot=128 * 512, oh=512, lse=A,
             ll=128, w=A, wb=ws):
        front = (ptable, pwidth, plen) if shared else ()
        fn = lib.dsnq_shared_prefix_latent_attention_fp8 if shared else lib.dsnq_paged_latent_attention_fp8
        return fn(B, H, K, P, DV, q, qt, qh, cache, pages, ps, lp, lr, scales, lds, *front, table, width, ldt, lens, scale,
                  out, ot, oh, lse, ll, w, wb, None)

    assert call(B=0) == OK
    assert call(B=-1) == INVALID and call(H=0) == INVALID and call(K=0) == INVALID and call(P=-64) == INVALID
    assert call(width=-1) == INVALID and call(ps=0) == INVALID and call(pages=0) == INVALID
    assert call(DV=640) == INVALID                            # a value wider than the latent
    assert call(K=448, DV=384) == UNSUPPORTED and call(K=640) == UNSUPPORTED and call(P=32) == UNSUPPORTED and call(P=128) == UNSUPPORTED
    assert call(DV=448) == UNSUPPORTED and call(H=1025) == UNSUPPORTED and call(B=8193) == UNSUPPORTED
    assert call(ps=60) == UNSUPPORTED and call(ps=4) == UNSUPPORTED
    assert call(lr=1 << 20, lp=1 << 21) == INVALID            # pages that overlap
    assert call(ps=8, lr=1 << 37, lp=1 << 41, width=1, ldt=1, pwidth=1) == UNSUPPORTED and call(qt=1 << 39) == UNSUPPORTED
    assert call(width=1 << 26, ldt=1 << 26) == UNSUPPORTED    # tokens of a request beyond int32
    assert call(scale=0.0) == INVALID and call(scale=-1.0) == INVALID and call(scale=float("nan")) == INVALID
    for name in ("q", "cache", "scales", "table", "lens", "out", "w"):
        assert call(**{name: None}) == INVALID, name
    assert call(qh=568) == INVALID and call(ot=504) == INVALID and call(ldt=15) == INVALID and call(ll=127) == INVALID
    assert call(lr=624) == INVALID and call(lp=64 * 640 - 16) == INVALID and call(lds=63) == INVALID
    assert call(wb=ws // 2) == INVALID                        # workspace too small
    assert call(q=A + 8) == MISALIGNED and call(lr=648, lp=64 * 648) == MISALIGNED and call(w=A + 8) == MISALIGNED
    assert call(lens=A + 2) == MISALIGNED and call(scales=A + 4) == MISALIGNED and call(lds=66) == MISALIGNED
    if shared:
        assert call(ptable=None) == INVALID and call(plen=None) == INVALID and call(pwidth=-1) == INVALID
        assert call(pwidth=1 << 26) == UNSUPPORTED
        assert call(plen=A + 2) == MISALIGNED and call(ptable=A + 1) == MISALIGNED


def test_workspace_queries(lib):
    """The split queries, and what the whole GPU's workers leave at most; with a
    prefix the parts grow with the batch too."""
    def size(B, H, DV=512, width=16, ps=64):
        return dsnq.paged_latent_attention_fp8_workspace_bytes(B, H, DV, width, ps)

    # Split queries: per 64 heads two e4m3 copies of 512 columns, 64 bf16 columns, a factor each.
    image = lambda rows: (2 * 4 + 1) * rows * 128 + 64 * 4
    assert size(0, 128) == 0
    assert size(1, 128, width=2) < size(1, 128) <= size(64, 128) - 63 * 2 * image(64)
    assert size(1000, 128) - size(64, 128) == 936 * 2 * image(64)
    assert size(1000, 128) < (43 << 20) + 2000 * image(64) and size(8192, 16, width=1000) < (43 << 20) + 8192 * image(16)

    def shared(B, H, pwidth=500, width=16):
        return dsnq.shared_prefix_latent_attention_fp8_workspace_bytes(B, H, 512, pwidth, width, 64)

    assert shared(0, 16) == 0 and shared(8, 16) < shared(64, 16) < shared(256, 16)
    # Two parts of DV floats for each pair of a request and a head (64 rows a part), and some for each worker.
    parts = 256 * 16 // 64 + 256 + 160
    assert shared(256, 16) < (parts + 2) * 64 * 516 * 4 + (256 * 16 // 64 + 256) * image(64) + 4096
    assert shared(8192, 1024) > 1 << 35                       # in 64 bits
    n = C.c_int64()
    q = lib.dsnq_shared_prefix_latent_attention_fp8_workspace_bytes
    assert q(4, 128, 500, 1, 16, 64, C.byref(n)) == UNSUPPORTED and q(-1, 128, 512, 1, 16, 64, None) == INVALID
    assert q(4, 128, 512, -1, 16, 64, None) == INVALID and q(1 << 40, 128, 512, 1, 16, 64, None) == UNSUPPORTED
    assert lib.dsnq_paged_latent_attention_fp8_workspace_bytes(4, 128, 512, 16, 60, None) == UNSUPPORTED


# --------------------------------------------------------------------- binding

class Recorder:
    """Stands for the library: every entry point records its call and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(dsnq, "lib", lambda: rec)
    monkeypatch.setattr(dsnq, "_stream", lambda stream, dev: 0)
    return rec


def z(*shape, dtype=BF, device="cpu"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def cache_args():
    return dict(cache=z(2, 16, 640, dtype=U8), scales=z(2, 16, dtype=F32))


def write_args():
    return dict(kv=z(4, 512), pe=z(4, 64), positions=z(4, dtype=I64), slots=z(4, dtype=I64), inv_freq=z(32, dtype=F64),
                **cache_args(), gamma=z(512), normalize=True)


def read_args():
    return dict(**cache_args(), latent_dim=512, block_table=z(4, 2, dtype=I32), row_starts=z(5, dtype=I32), rows=9, first=z(4, dtype=I32),
                out=z(9, 576))


def attention_args():
    return dict(q=z(4, 8, 576), **cache_args(), block_table=z(4, 2, dtype=I32), seq_lens=z(4, dtype=I32), v_dim=512, scale=0.1,
                out=z(4, 8, 512), lse=z(4, 8, dtype=F32), workspace=z(1 << 20, dtype=U8))


def shared_args():
    return dict(**attention_args(), prefix_table=z(7, dtype=I32), prefix_len=z(1, dtype=I32))


OPS = {"write": (dsnq.latent_cache_write_fp8, write_args), "read": (dsnq.latent_cache_read_fp8, read_args),
       "attention": (dsnq.paged_latent_attention_fp8, attention_args), "shared": (dsnq.shared_prefix_latent_attention_fp8, shared_args)}


def pointers(a):
    return {k: v.data_ptr() for k, v in a.items() if torch.is_tensor(v)}


def test_write_hands_on(library):
    a = write_args()
    got = dsnq.latent_cache_write_fp8(**a, layout="half", rope_scale=1.5)
    assert got[0] is a["cache"] and got[1] is a["scales"]
    p = pointers(a)
    assert library.calls == [("dsnq_latent_cache_write_fp8", (
        4, 512, 64, p["kv"], 512, p["pe"], 64, 1, p["gamma"], 1e-6, p["positions"], p["inv_freq"], 512, 64, dsnq.ROPE_HALF, 1.5,
        p["slots"], p["cache"], 2, 16, 16 * 640, 640, p["scales"], 16, 0))]
    library.calls.clear()
    dsnq.latent_cache_write_fp8(a["kv"], None, a["positions"], a["slots"], a["inv_freq"], z(2, 16, 512, dtype=U8), a["scales"])
    c = library.calls[0][1]
    assert c[:9] == (4, 512, 0, p["kv"], 512, None, 0, 0, None) and c[12] == 448


def test_read_hands_on(library):
    a = read_args()
    assert dsnq.latent_cache_read_fp8(**a) is a["out"]
    p = pointers(a)
    assert library.calls == [("dsnq_latent_cache_read_fp8", (
        4, 9, 512, 64, p["cache"], 2, 16, 16 * 640, 640, p["scales"], 16, p["block_table"], 2, 2, p["row_starts"], p["first"], p["out"],
        576, 0))]
    library.calls.clear()
    a.update(first=None, out=None)
    assert dsnq.latent_cache_read_fp8(**a).shape == (9, 576) and library.calls[0][1][15] is None


def test_attention_hands_on(library):
    a = attention_args()
    out, lse = dsnq.paged_latent_attention_fp8(**a)
    assert out is a["out"] and lse is a["lse"]
    p = pointers(a)
    head = (4, 8, 512, 64, 512, p["q"], 8 * 576, 576, p["cache"], 2, 16, 16 * 640, 640, p["scales"], 16)
    tail = (p["block_table"], 2, 2, p["seq_lens"], 0.1, p["out"], 8 * 512, 512, p["lse"], 8, p["workspace"], 1 << 20, 0)
    assert library.calls == [("dsnq_paged_latent_attention_fp8", head + tail)]
    library.calls.clear()
    s = {**a, **{k: v for k, v in shared_args().items() if k.startswith("prefix")}}
    dsnq.shared_prefix_latent_attention_fp8(**s)
    assert library.calls == [("dsnq_shared_prefix_latent_attention_fp8",
                              head + (s["prefix_table"].data_ptr(), 7, s["prefix_len"].data_ptr()) + tail)]


CACHE_REFUSED = [
    (dict(cache=z(2, 16, 640)), TypeError, "cache must be torch.uint8"),
    (dict(cache=z(32, 640, dtype=U8)), ValueError, "cache must have 3 dimensions"),
    (dict(cache=z(2, 640, 16, dtype=U8).transpose(1, 2)), ValueError, "cache must have contiguous rows"),
    (dict(scales=z(2, 16)), TypeError, "scales must be torch.float32"),
    (dict(scales=z(32, dtype=F32)), ValueError, "scales must have 2 dimensions"),
    (dict(scales=z(16, 2, dtype=F32).t()), ValueError, "scales must have contiguous rows"),
    (dict(scales=z(2, 15, dtype=F32)), ValueError, "scales has shape"),
    (dict(scales=z(3, 16, dtype=F32)), ValueError, "scales has shape"),
]
REFUSED = [(op, *r) for op in OPS for r in CACHE_REFUSED] + [
    ("write", dict(kv=z(4, 512, dtype=F32)), TypeError, "kv must be torch.bfloat16"),
    ("write", dict(kv=z(512, 4).t()), ValueError, "kv must have contiguous rows"),
    ("write", dict(kv=z(4, 448)), ValueError, "cache rows have 640 bytes, kv and pe make 576"),
    ("write", dict(pe=z(3, 64)), ValueError, "pe has 3 rows, kv 4"),
    ("write", dict(pe=None), ValueError, "cache rows have 640 bytes, kv and pe make 512"),
    ("write", dict(positions=z(3, dtype=I64)), ValueError, "positions must be contiguous with 4 elements"),
    ("write", dict(slots=z(4, dtype=I32)), TypeError, "slots must be torch.int64"),
    ("write", dict(inv_freq=z(32, dtype=F32)), TypeError, "inv_freq must be torch.float64"),
    ("write", dict(gamma=z(576)), ValueError, "gamma must be contiguous with 512 elements"),
    ("write", dict(layout=2), ValueError, "unknown rotary layout"),
    ("read", dict(latent_dim=0), ValueError, "do not hold 0 codes"),
    ("read", dict(latent_dim=511), ValueError, "do not hold 511 codes"),
    ("read", dict(latent_dim=700), ValueError, "do not hold 700 codes"),
    ("read", dict(block_table=z(4, 2, dtype=I64)), TypeError, "block_table must be torch.int32"),
    ("read", dict(row_starts=z(4, dtype=I32)), ValueError, "row_starts must be contiguous with 5 elements"),
    ("read", dict(row_starts=z(5, dtype=I64)), TypeError, "row_starts must be torch.int32"),
    ("read", dict(first=z(5, dtype=I32)), ValueError, "first must be contiguous with 4 elements"),
    ("read", dict(out=z(9, 512)), ValueError, "out has shape"),
    ("read", dict(out=z(8, 576)), ValueError, "out has shape"),
    ("read", dict(out=z(9, 576, dtype=F32)), TypeError, "out must be torch.bfloat16"),
]
for _op in ("attention", "shared"):
    REFUSED += [
        (_op, dict(q=z(4, 8, 576, dtype=F32)), TypeError, "q must be torch.bfloat16"),
        (_op, dict(q=z(4, 8, 656)), ValueError, "cache rows of 640 bytes do not fit q's 656 columns"),
        (_op, dict(q=z(4, 8, 320)), ValueError, "cache rows of 640 bytes do not fit q's 320 columns"),
        (_op, dict(q=z(8, 576)), ValueError, "q must have 3 dimensions"),
        (_op, dict(block_table=z(3, 2, dtype=I32)), ValueError, "block_table has 3 rows for 4 requests"),
        (_op, dict(seq_lens=z(4, dtype=I64)), TypeError, "seq_lens must be torch.int32"),
        (_op, dict(seq_lens=z(3, dtype=I32)), ValueError, "seq_lens must be contiguous with 4 elements"),
        (_op, dict(out=z(4, 8, 576)), ValueError, "out has shape"),
        (_op, dict(out=z(4, 8, 512, dtype=F32)), TypeError, "out must be torch.bfloat16"),
        (_op, dict(lse=z(4, 4, dtype=F32)), ValueError, "lse has shape"),
        (_op, dict(workspace=z(8, dtype=F32)), TypeError, "workspace must be torch.uint8"),
    ]
REFUSED += [
    ("shared", dict(prefix_table=z(7, dtype=I64)), TypeError, "prefix_table must be torch.int32"),
    ("shared", dict(prefix_table=z(1, 7, dtype=I32)), ValueError, "prefix_table must have 1 dimensions"),
    ("shared", dict(prefix_table=z(14, dtype=I32)[::2]), ValueError, "prefix_table must be contiguous"),
    ("shared", dict(prefix_table=None), TypeError, "prefix_table must be a tensor"),
    ("shared", dict(prefix_len=z(2, dtype=I32)), ValueError, "prefix_len must be contiguous with 1 elements"),
    ("shared", dict(prefix_len=z(1, dtype=I64)), TypeError, "prefix_len must be torch.int32"),
]


@pytest.mark.parametrize("op,bad,error,why", REFUSED, ids=[f"{r[0]}-{next(iter(r[1]))}-{i}" for i, r in enumerate(REFUSED)])
def test_wrong_arguments_are_refused_by_name(library, op, bad, error, why):
    fn, args = OPS[op]
    a = args()
    a.update(bad)
    with pytest.raises(error, match=why.replace("[", r"\[")):
        fn(**a)
    assert library.calls == []


@pytest.mark.parametrize("op,name", [(op, k) for op, (_, args) in OPS.items() for k, v in args().items() if torch.is_tensor(v)])
def test_tensors_of_another_device_are_refused_by_name(library, op, name):
    """Each tensor in turn on another device than the one the others are on."""
    fn, args = OPS[op]
    a = args()
    a[name] = a[name].to("meta")
    first = next(iter(a))                                    # the tensor that names the call's device
    with pytest.raises(ValueError, match=r"is on cpu, expected meta" if name == first else f"{name} is on meta, expected cpu"):
        fn(**a)
    assert library.calls == []


def test_cpu_tensors_are_refused():
    for fn, args in OPS.values():
        with pytest.raises(ValueError, match="must be CUDA tensors"):
            fn(**args())


def test_workspaces_are_as_large_as_stated():
    """The header's and the binding's account of the workspaces, for few and many heads and requests."""
    up = lambda a, b: -(-a // b)
    for B in (1, 3, 64, 256, 1000, 8192):
        for H in (1, 6, 16, 48, 64, 100, 128, 1024):
            for DV in (128, 512):
                for pwidth, width in ((20, 4), (500, 16), (40000, 2000)):
                    groups = up(H, 64)
                    for shared in (False, True):
                        if shared:
                            got = dsnq.shared_prefix_latent_attention_fp8_workspace_bytes(B, H, DV, pwidth, width, 64)
                            sets = B * groups + up(B * up(H, 4) * 4, 64)
                            least, most = sets * (73_000 + 256 * DV) if sets > 320 else 0, sets * (75_000 + 256 * DV + 512) + (54 << 20)
                        else:
                            got = dsnq.paged_latent_attention_fp8_workspace_bytes(B, H, DV, width, 64)
                            rows = B * up(H, 16) * 16
                            least, most = rows * 1152, B * H * 1300 + B * (groups * 256 + 16 * 1200) + (42 << 20) + (1 << 19)
                        assert least <= got <= most, (B, H, DV, pwidth, width, shared, got, least, most)
