"""Which requests of the paged latent attention are cut over workers (the
workspace begins with each worker's first request and its first tile there),
kept workspaces that are given back, and a lone row of the cache write."""

import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cuts(lens, H, width=None):
    """How many workers begin inside a request, and how many have work."""
    pages = sum(-(-n // 64) for n in lens)
    width = width or max(-(-n // 64) for n in lens)
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = torch.randn(pages, 64, 576, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // 64)
        table[b, :k] = torch.arange(at, at + k, device=DEV)
        at += k
    q = torch.randn(len(lens), H, 576, generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.full((dsnq.paged_latent_attention_workspace_bytes(len(lens), H, 512, width, 64),), 255, dtype=torch.uint8, device=DEV)
    dsnq.paged_latent_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 512, 0.05, workspace=ws)
    assert dsnq.debug_status() == 0
    groups = -(-H // 64)
    workers = min(torch.cuda.get_device_properties(0).multi_processor_count // groups, len(lens) * width)
    first = ws[:8 * workers].view(torch.int32).view(-1, 2).cpu()
    assert bool((first[:, 0] >= 0).all()) and bool((first[:, 0] <= len(lens)).all())
    live = first[first[:, 0] < len(lens)]
    return int((live[:, 1] > 0).sum()), len(set(map(tuple, live.tolist())))


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("width", [None, 200])
def test_a_short_request_on_an_idle_gpu_is_cut(H, width):
    """512 tokens, 8 tiles: a worker takes one of them, two at most, whether
    the table is just long enough or much longer (one worker took them in turn:
    22 us instead of 12.5 at 64 heads and more).  With a table of 8 pages there
    are 8 workers for 9 units, the tiles and one that stands for the request:
    two begin at tile 0, so 6 begin inside."""
    inside, working = cuts([512], H, width)
    assert (inside, working) == ((6, 7) if width is None else (7, 8))
    inside, _ = cuts([450, 512, 300], H, width)
    assert inside > 10


def test_one_or_two_tiles_stay_whole():
    assert cuts([128], 128)[0] == 0 and cuts([1, 64, 100], 16)[0] == 0


def test_requests_of_about_a_workers_share_stay_whole():
    """64 of 1000 tokens at 128 heads: 16 tiles each, a share is 14."""
    inside, working = cuts([1000] * 64, 128)
    assert (inside, working) == (0, 64)
    assert cuts([500] * 16, 128)[0] == 0


def test_a_long_request_among_short_ones_is_cut():
    inside, working = cuts([9000] + [100] * 20, 64)
    assert inside > 100


def test_workspaces_may_be_released_between_calls():
    """Given back while a call still runs, and between a capture and its
    replays: the memory goes to later work of the same stream only."""
    lens, H = [3000, 70, 900], 64
    g = torch.Generator(device=DEV).manual_seed(2)
    cache = torch.randn(70, 64, 576, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.randperm(70, generator=g, device=DEV)[:70].to(torch.int32).view(1, 70)[:, :47].expand(3, 47).contiguous()
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn(3, H, 576, generator=g, device=DEV).to(torch.bfloat16)
    want = dsnq.paged_latent_attention(q, cache, table, n, 512, 0.05)
    junk = []
    for _ in range(20):
        got = dsnq.paged_latent_attention(q, cache, table, n, 512, 0.05)
        dsnq.release_workspaces()
        junk.append(torch.full((1 << 20,), float("nan"), device=DEV))        # may take the memory
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dsnq.paged_latent_attention(q, cache, table, n, 512, 0.05)
    dsnq.release_workspaces()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert dsnq.debug_status() == 0


def test_a_lone_row_of_a_buffer_with_an_odd_stride():
    """One kv row of a buffer whose rows are 2113 apart: the stride is never used."""
    row = torch.randn(1, 2113, device=DEV).to(torch.bfloat16)
    cache = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device=DEV)
    i64 = lambda x: torch.tensor(x, device=DEV)
    f = torch.zeros(0, dtype=torch.float64, device=DEV)
    dsnq.latent_cache_write(row[:, 1536:2048], row[:, 2048:2112], i64([5]), i64([11]), f, cache)
    assert torch.equal(cache[1, 3], row[0, 1536:2112]) and int((cache != 0).any(-1).sum()) == 1
    assert dsnq.debug_status() == 0
