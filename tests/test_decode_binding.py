"""The binding of the decode-step operators without a GPU: what it hands to
the library, and that each wrong argument is refused by name before the
library is reached.  The library is a recorder here, and the stream's check
(which refuses every CPU tensor) is out of the way."""

import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq

I32, I64, BF, F32, F64, U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.float64, torch.uint8


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


def head_args():
    return dict(x=z(4, 3, 64), positions=z(4, dtype=I64), inv_freq=z(32, dtype=F64), gamma=z(64), out=z(4, 3, 64))


def write_args():
    return dict(kv=z(4, 512), pe=z(4, 64), positions=z(4, dtype=I64), slots=z(4, dtype=I64), inv_freq=z(32, dtype=F64),
                cache=z(2, 16, 576), gamma=z(512), normalize=True)


def attention_args():
    return dict(q=z(4, 8, 576), cache=z(2, 16, 576), block_table=z(4, 2, dtype=I32), seq_lens=z(4, dtype=I32), v_dim=512, scale=0.1,
                out=z(4, 8, 512), lse=z(4, 8, dtype=F32), workspace=z(1 << 20, dtype=U8))


def extend_args():
    return dict(seq_lens=z(4, dtype=I32), new_tokens=z(4, dtype=I32), free_pages=z(7, dtype=I32), block_table=z(4, 2, dtype=I32),
                page_size=16, rows=9,
                out=(z(4, dtype=I32), z(5, dtype=I32), z(9, dtype=I64), z(9, dtype=I64), z(2, dtype=I32)))


OPS = {"head": (dsnq.head_rmsnorm_rope, head_args, "dsnq_head_rmsnorm_rope"),
       "write": (dsnq.latent_cache_write, write_args, "dsnq_latent_cache_write"),
       "attention": (dsnq.paged_latent_attention, attention_args, "dsnq_paged_latent_attention"),
       "extend": (dsnq.extend_block_tables, extend_args, "dsnq_extend_block_tables")}


# ------------------------------------------------------------ what is handed on

def test_head_norm_rope_hands_on(library):
    a = head_args()
    assert dsnq.head_rmsnorm_rope(**a, rope_scale=1.5, inverse=True, layout="half") is a["out"]
    (name, c), = library.calls
    p = {k: v.data_ptr() for k, v in a.items()}
    assert name == "dsnq_head_rmsnorm_rope"
    assert c == (4, 3, 64, p["x"], 192, 64, 1, p["gamma"], 1e-6, p["positions"], p["inv_freq"], 0, 64, dsnq.ROPE_HALF, 1.5, 1,
                 p["out"], 192, 64, 0)


def test_cache_write_hands_on(library):
    a = write_args()
    assert dsnq.latent_cache_write(**a) is a["cache"]
    p = {k: v.data_ptr() for k, v in a.items() if k != "normalize"}
    assert library.calls == [("dsnq_latent_cache_write", (
        4, 512, 64, p["kv"], 512, p["pe"], 64, 1, p["gamma"], 1e-6, p["positions"], p["inv_freq"], 512, 64,
        dsnq.ROPE_INTERLEAVED, 1.0, p["slots"], p["cache"], 2, 16, 16 * 576, 576, 0))]
    library.calls.clear()
    dsnq.latent_cache_write(a["kv"], None, a["positions"], a["slots"], a["inv_freq"], z(2, 16, 512))
    c = library.calls[0][1]
    assert c[:9] == (4, 512, 0, p["kv"], 512, None, 0, 0, None) and c[12] == 448


def test_attention_hands_on(library):
    a = attention_args()
    out, lse = dsnq.paged_latent_attention(**a)
    assert out is a["out"] and lse is a["lse"]
    p = {k: v.data_ptr() for k, v in a.items() if torch.is_tensor(v)}
    assert library.calls == [("dsnq_paged_latent_attention", (
        4, 8, 576, 512, p["q"], 8 * 576, 576, p["cache"], 2, 16, 16 * 576, 576, p["block_table"], 2, 2, p["seq_lens"], 0.1,
        p["out"], 8 * 512, 512, p["lse"], 8, p["workspace"], 1 << 20, 0))]


def test_extend_hands_on(library):
    a = extend_args()
    assert dsnq.extend_block_tables(**a) == a["out"]
    p = {k: v.data_ptr() for k, v in a.items() if torch.is_tensor(v)}
    assert library.calls == [("dsnq_extend_block_tables", (
        4, 9, 16, p["seq_lens"], p["new_tokens"], p["free_pages"], 7, p["block_table"], 2, 2,
        *[t.data_ptr() for t in a["out"]], 0))]
    library.calls.clear()
    a["new_tokens"] = None
    dsnq.extend_block_tables(**a)
    assert library.calls[0][1][4] is None


def test_a_lone_row_has_no_stride(library):
    """One row of a buffer whose rows are no multiple of 8 apart: the stride is
    never used, so it must not reach the library, which would refuse it."""
    a = write_args()
    row = z(1, 2113)
    a.update(kv=row[:, :512], pe=row[:, 512:576], positions=a["positions"][:1], slots=a["slots"][:1])
    dsnq.latent_cache_write(**a)
    c = library.calls[0][1]
    assert c[0] == 1 and c[4] == 512 and c[6] == 64


# ------------------------------------------------------------------- refusals

def out_with(i, t):
    o = list(extend_args()["out"])
    o[i] = t
    return tuple(o)


REFUSED = [
    ("head", dict(x=z(4, 3, 64, dtype=F32)), TypeError, "x must be torch.bfloat16"),
    ("head", dict(x=z(4, 3, 64, dtype=torch.float16)), TypeError, "x must be torch.bfloat16"),
    ("head", dict(x=z(3, 64)), ValueError, "x must have 3 dimensions"),
    ("head", dict(x=z(4, 64, 3).transpose(1, 2)), ValueError, "x must have contiguous rows"),
    ("head", dict(positions=z(4, dtype=I32)), TypeError, "positions must be torch.int64"),
    ("head", dict(positions=z(3, dtype=I64)), ValueError, "positions must be contiguous with 4 elements"),
    ("head", dict(positions=z(5, dtype=I64)), ValueError, "positions must be contiguous with 4 elements"),
    ("head", dict(positions=z(8, dtype=I64)[::2]), ValueError, "positions must be contiguous with 4 elements"),
    ("head", dict(positions=z(4, 1, dtype=I64)), ValueError, "positions must have 1 dimensions"),
    ("head", dict(inv_freq=z(32, dtype=F32)), TypeError, "inv_freq must be torch.float64"),
    ("head", dict(inv_freq=z(32, 1, dtype=F64)), ValueError, "inv_freq must have 1 dimensions"),
    ("head", dict(inv_freq=z(64, dtype=F64)[::2]), ValueError, "inv_freq must be contiguous"),
    ("head", dict(gamma=z(32)), ValueError, "gamma must be contiguous with 64 elements"),
    ("head", dict(gamma=z(64, dtype=F32)), TypeError, "gamma must be torch.bfloat16"),
    ("head", dict(out=z(4, 3, 32)), ValueError, "out has shape"),
    ("head", dict(out=z(3, 3, 64)), ValueError, "out has shape"),
    ("head", dict(out=z(4, 2, 64)), ValueError, "out has shape"),
    ("head", dict(out=z(4, 3, 64, dtype=F32)), TypeError, "out must be torch.bfloat16"),
    ("head", dict(layout="other"), ValueError, "unknown rotary layout"),
    ("write", dict(kv=z(4, 512, dtype=F32)), TypeError, "kv must be torch.bfloat16"),
    ("write", dict(kv=z(512)), ValueError, "kv must have 2 dimensions"),
    ("write", dict(kv=z(512, 4).t()), ValueError, "kv must have contiguous rows"),
    ("write", dict(kv=z(4, 448)), ValueError, "cache rows have 576 columns, kv and pe 512"),
    ("write", dict(pe=z(3, 64)), ValueError, "pe has 3 rows, kv 4"),
    ("write", dict(pe=z(4, 64, dtype=F32)), TypeError, "pe must be torch.bfloat16"),
    ("write", dict(pe=None), ValueError, "cache rows have 576 columns, kv and pe 512"),
    ("write", dict(positions=z(3, dtype=I64)), ValueError, "positions must be contiguous with 4 elements"),
    ("write", dict(positions=z(4, dtype=I32)), TypeError, "positions must be torch.int64"),
    ("write", dict(slots=z(4, dtype=I32)), TypeError, "slots must be torch.int64"),
    ("write", dict(slots=z(3, dtype=I64)), ValueError, "slots must be contiguous with 4 elements"),
    ("write", dict(inv_freq=z(32, dtype=F32)), TypeError, "inv_freq must be torch.float64"),
    ("write", dict(cache=z(2, 16, 512)), ValueError, "cache rows have 512 columns, kv and pe 576"),
    ("write", dict(cache=z(32, 576)), ValueError, "cache must have 3 dimensions"),
    ("write", dict(cache=z(2, 16, 576, dtype=F32)), TypeError, "cache must be torch.bfloat16"),
    ("write", dict(gamma=z(576)), ValueError, "gamma must be contiguous with 512 elements"),
    ("write", dict(layout=2), ValueError, "unknown rotary layout"),
    ("attention", dict(q=z(4, 8, 576, dtype=F32)), TypeError, "q must be torch.bfloat16"),
    ("attention", dict(q=z(4, 8, 512)), ValueError, "cache rows have 576 columns, q 512"),
    ("attention", dict(q=z(8, 576)), ValueError, "q must have 3 dimensions"),
    ("attention", dict(cache=z(2, 16, 576, dtype=torch.float16)), TypeError, "cache must be torch.bfloat16"),
    ("attention", dict(cache=z(2, 576, 16).transpose(1, 2)), ValueError, "cache must have contiguous rows"),
    ("attention", dict(block_table=z(4, 2, dtype=I64)), TypeError, "block_table must be torch.int32"),
    ("attention", dict(block_table=z(3, 2, dtype=I32)), ValueError, "block_table has 3 rows for 4 requests"),
    ("attention", dict(block_table=z(2, 4, dtype=I32).t()), ValueError, "block_table must have contiguous rows"),
    ("attention", dict(seq_lens=z(4, dtype=I64)), TypeError, "seq_lens must be torch.int32"),
    ("attention", dict(seq_lens=z(3, dtype=I32)), ValueError, "seq_lens must be contiguous with 4 elements"),
    ("attention", dict(out=z(4, 8, 576)), ValueError, "out has shape"),
    ("attention", dict(out=z(4, 7, 512)), ValueError, "out has shape"),
    ("attention", dict(out=z(4, 8, 512, dtype=F32)), TypeError, "out must be torch.bfloat16"),
    ("attention", dict(lse=z(4, 4, dtype=F32)), ValueError, "lse has shape"),
    ("attention", dict(lse=z(4, 8)), TypeError, "lse must be torch.float32"),
    ("attention", dict(lse=z(8, 4, dtype=F32).t()), ValueError, "lse must have contiguous rows"),
    ("attention", dict(workspace=z(8, dtype=F32)), TypeError, "workspace must be torch.uint8"),
    ("attention", dict(workspace=z(8, 2, dtype=U8)), ValueError, "workspace must have 1 dimensions"),
    ("extend", dict(seq_lens=z(4, dtype=I64)), TypeError, "seq_lens must be torch.int32"),
    ("extend", dict(seq_lens=z(4, 1, dtype=I32)), ValueError, "seq_lens must have 1 dimensions"),
    ("extend", dict(seq_lens=z(3, dtype=I32)), ValueError, "block_table has 4 rows for 3 requests"),
    ("extend", dict(new_tokens=z(2, dtype=I32)), ValueError, "new_tokens must be contiguous with 4 elements"),
    ("extend", dict(new_tokens=z(4, dtype=I64)), TypeError, "new_tokens must be torch.int32"),
    ("extend", dict(free_pages=z(14, dtype=I32)[::2]), ValueError, "free_pages must be contiguous"),
    ("extend", dict(free_pages=z(7, dtype=I64)), TypeError, "free_pages must be torch.int32"),
    ("extend", dict(block_table=z(4, 2, dtype=I64)), TypeError, "block_table must be torch.int32"),
    ("extend", dict(block_table=z(2, 4, dtype=I32).t()), ValueError, "block_table must have contiguous rows"),
    ("extend", dict(rows=10), ValueError, "positions must be contiguous with 10 elements"),
    ("extend", dict(out=out_with(0, z(3, dtype=I32))), ValueError, "new_lens must be contiguous with 4 elements"),
    ("extend", dict(out=out_with(1, z(4, dtype=I32))), ValueError, "row_starts must be contiguous with 5 elements"),
    ("extend", dict(out=out_with(2, z(9, dtype=I32))), TypeError, "positions must be torch.int64"),
    ("extend", dict(out=out_with(3, z(8, dtype=I64))), ValueError, "slots must be contiguous with 9 elements"),
    ("extend", dict(out=out_with(4, z(1, dtype=I32))), ValueError, "counts must be contiguous with 2 elements"),
]


@pytest.mark.parametrize("op,bad,error,why", REFUSED, ids=[f"{r[0]}-{next(iter(r[1]))}-{i}" for i, r in enumerate(REFUSED)])
def test_wrong_arguments_are_refused_by_name(library, op, bad, error, why):
    fn, args, _ = OPS[op]
    a = args()
    a.update(bad)
    with pytest.raises(error, match=why.replace("[", r"\[")):
        fn(**a)
    assert library.calls == []


@pytest.mark.parametrize("op,name", [(op, k) for op, (_, args, _) in OPS.items() for k, v in args().items() if torch.is_tensor(v)])
def test_tensors_of_another_device_are_refused_by_name(library, op, name):
    """Each tensor in turn on another device than the one the others are on."""
    fn, args, _ = OPS[op]
    a = args()
    a[name] = a[name].to("meta")
    first = next(iter(a))                                    # the tensor that names the call's device
    with pytest.raises(ValueError, match=r"is on cpu, expected meta" if name == first else f"{name} is on meta, expected cpu"):
        fn(**a)
    assert library.calls == []


# ------------------------------------------------------------- kept workspaces

CPU = torch.device("cpu")


@pytest.fixture
def eager(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    dsnq.release_workspaces()
    yield
    dsnq.release_workspaces()


def test_a_stream_in_use_keeps_its_workspace(eager):
    """The four streams used last keep theirs: one that every other call uses
    is never among those that lose it, the others go in turn."""
    mine = dsnq._workspace(100, CPU, None, 1)
    others = {}
    for h in range(2, 12):
        others[h] = dsnq._workspace(100, CPU, None, h)
        assert dsnq._workspace(100, CPU, None, 1) is mine
    assert dsnq._workspace(100, CPU, None, 11) is others[11]
    assert dsnq._workspace(100, CPU, None, 10) is others[10]
    assert dsnq._workspace(100, CPU, None, 9) is others[9]
    assert dsnq._workspace(100, CPU, None, 8) is not others[8]


def test_workspaces_of_devices_are_counted_apart(eager, monkeypatch):
    """Five devices with a stream each: all keep theirs."""
    class Device(str):
        index = property(lambda self: int(self[4:]))

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: empty(n, dtype=dtype))
    devs = [Device(f"cuda{i}") for i in range(5)]
    kept = [dsnq._workspace(10, d, None, 7) for d in devs]
    assert all(dsnq._workspace(10, d, None, 7) is t for d, t in zip(devs, kept))
    assert len({t.data_ptr() for t in kept}) == 5


def test_a_workspace_grows_and_is_given_back(eager):
    import gc
    import weakref
    small = dsnq._workspace(10, CPU, None, 1)
    assert dsnq._workspace(5, CPU, None, 1) is small
    large = dsnq._workspace(20, CPU, None, 1)
    assert large is not small and large.numel() == 20 and dsnq._workspace(10, CPU, None, 1) is large
    ref = weakref.ref(large)
    del small, large
    dsnq.release_workspaces()
    gc.collect()
    assert ref() is None


def test_captures_and_explicit_streams_keep_none(eager, monkeypatch):
    monkeypatch.setattr(dsnq, "_new", lambda shape, dtype, dev, stream: torch.empty(shape, dtype=dtype, device=dev))
    assert dsnq._workspace(10, CPU, 5, 5) is not dsnq._workspace(10, CPU, 5, 5)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert dsnq._workspace(10, CPU, None, 5) is not dsnq._workspace(10, CPU, None, 5)
    assert not dsnq._kept.__dict__
