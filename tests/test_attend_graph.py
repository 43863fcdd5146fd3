"""pkv_attend and pkv_attend_fp8 captured into a graph and replayed: the counters
that join a row's parts are told apart by the call's number, which a replay
repeats, so a captured call leaves none of it behind."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import to_device
from workloads import make_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_lens", [([17, 64, 100, 255], [1, 1, 1, 1]), ([400, 3, 2090, 16], [1, 3, 1, 1]),
                                         ([300, 700, 90, 1200], [1, 40, 1, 300])])
def test_replays_with_new_lengths(pkvlib, lens, q_lens, fp8):
    pkv.get_last_error()
    b = make_batch(lens, q_lens, 32, 8, seed=91, device="cuda")
    meta = to_device(b)
    if fp8:
        shape = b.k_cache.shape
        e4m3 = lambda x: (x.float().clamp(-4, 4) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.full(shape[:3], 121, device="cuda", dtype=torch.uint8)
        pools, call, size = [e4m3(b.k_cache), e4m3(b.v_cache), scale, scale], pkv.attend_fp8, pkv.workspace_size_fp8
    else:
        pools, call, size = [b.k_cache, b.v_cache], pkv.attend, pkv.workspace_size
    lens_now, tail = meta["seq_lens"].clone(), (meta["query_start_loc"], b.scale)
    need = size(pkv.make_desc(pools[0], 32, meta["block_tables"].shape[1]), b.B, b.q.shape[0])
    ws = torch.full((need,), 255, device="cuda", dtype=torch.uint8)
    out = torch.empty_like(b.q)
    call(b.q, *pools, meta["block_tables"], lens_now, *tail, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(b.q, *pools, meta["block_tables"], lens_now, *tail, out=out, workspace=ws)
    noise = torch.empty(2, 1 << 26, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    rng = np.random.default_rng(91)
    counters = ws[:b.q.shape[0] * 8 * 8].view(torch.int64)  # a word a (row, kv head): four query heads share one
    for _ in range(30):
        L = np.array([rng.integers(n, top, endpoint=True) for n, top in zip(q_lens, lens)], np.int32)
        lens_now.copy_(torch.from_numpy(L))
        want = call(b.q, *pools, meta["block_tables"], lens_now.clone(), *tail)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            noise[0].copy_(noise[1])
        for _ in range(3):  # behind one another, as a decode loop replays
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert not bool(counters.any())
    assert pkv.get_last_error() == 0
