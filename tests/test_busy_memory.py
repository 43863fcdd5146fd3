"""pkv_attend and pkv_attend_fp8 beside another stream's copies: the same bits
call after call.  In these batches the last CTA of the split-KV kernel has work
for a few of its warps only, so that other kernels' blocks find room beside it
and its warps' reads of shared memory queue behind theirs."""

import numpy as np
import pytest
import torch

import oracle.pkv_oracle as O
import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits, compare, to_device
from workloads import make_batch

pytestmark = pytest.mark.gpu

WARPS = 12  # of a CTA


def batch(hq, hkv, last, seed):
    """A decode batch whose last CTA has ``last`` warps with work."""
    warps = WARPS * torch.cuda.get_device_properties(0).multi_processor_count
    items = hkv * (hq // hkv // min(4, hq // hkv))  # page reads a row
    for s in range(seed, seed + 5000):
        lens = np.random.default_rng(s).integers(1, 2500, size=83, endpoint=True)
        units = int((-(-lens // 16)).sum()) * items
        chunk = max(2, -(-units // warps))
        if (-(-units // chunk) - 1) % WARPS + 1 == last:
            return make_batch(lens.tolist(), [1] * 83, hq, hkv, seed=s, device="cuda")
    raise AssertionError("no such batch")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,last", [(32, 2, 4), (32, 8, 2), (16, 1, 3), (8, 8, 1)])
def test_the_same_bits_beside_copies(pkvlib, hq, hkv, last, fp8):
    pkv.get_last_error()
    b = batch(hq, hkv, last, 80)
    meta = to_device(b)
    tail = (meta["block_tables"], meta["seq_lens"], meta["query_start_loc"], b.scale)
    rows = np.flatnonzero(b.seq_lens >= 100)[-3:]  # (a decode batch: row = sequence)
    if fp8:
        shape = b.k_cache.shape
        pools = [torch.zeros(shape, device="cuda", dtype=torch.uint8) for _ in range(2)]
        pools += [torch.zeros(shape[:3], device="cuda", dtype=torch.uint8) for _ in range(2)]
        slots = torch.arange(shape[0] * 16, device="cuda")
        token = lambda x: x.transpose(1, 2).reshape(-1, shape[1], 128).contiguous()
        pkv.write_fp8(token(b.k_cache), token(b.v_cache), slots, *pools)
        call, size = pkv.attend_fp8, pkv.workspace_size_fp8
        host = [p.cpu().numpy() for p in pools]
        want = O.attend_fp8(bits(b.q), *host, b.block_tables, b.seq_lens, b.query_start_loc, b.scale, hq, hkv, 16,
                            rows=rows)
    else:
        pools, call, size = [b.k_cache, b.v_cache], pkv.attend, pkv.workspace_size
        want = O.attend(bits(b.q), bits(b.k_cache), bits(b.v_cache), b.block_tables, b.seq_lens, b.query_start_loc,
                        b.scale, hq, hkv, 16, rows=rows)
    ws = torch.empty(size(pkv.make_desc(pools[0], hq, tail[0].shape[1]), b.B, b.B), device="cuda", dtype=torch.uint8)
    first = call(b.q, *pools, *tail, workspace=ws, max_query_len=1)
    compare(first, want, rows=rows)
    noise = torch.empty(2, 1 << 26, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    for _ in range(25):
        outs = []
        for _ in range(20):
            with torch.cuda.stream(side):
                noise[0].copy_(noise[1])
            outs.append(call(b.q, *pools, *tail, workspace=ws, max_query_len=1))
        torch.cuda.synchronize()
        assert all(torch.equal(first.view(torch.int16), o.view(torch.int16)) for o in outs)
    assert pkv.get_last_error() == 0
