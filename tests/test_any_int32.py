"""pkv_attend and pkv_attend_fp8 with lengths and query starts that no batch has:
any int32 in their place is flagged, its sequence skipped and its neighbours
right (a length near 2^31 used to pass the table-width check by overflow)."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import to_device
from workloads import make_batch

pytestmark = pytest.mark.gpu

TOP = 2**31 - 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 40, 1], [1, 3, 40]])
def test_any_int32_as_length_or_query_start(pkvlib, q_lens, fp8):
    b = make_batch([100, 50, 60], q_lens, 32, 8, seed=51, device="cuda")
    meta = to_device(b)
    if fp8:
        pools = []
        for x in (b.k_cache, b.v_cache):
            pools.append(torch.randint(0, 0x70, x.shape, device="cuda", dtype=torch.uint8))
        pools += [torch.full(b.k_cache.shape[:3], 120, device="cuda", dtype=torch.uint8) for _ in range(2)]
    else:
        pools = [b.k_cache, b.v_cache]
    call = pkv.attend_fp8 if fp8 else pkv.attend

    def run(lens, starts):
        out = torch.full_like(b.q, 7.0)
        call(b.q, *pools, meta["block_tables"], torch.from_numpy(lens).cuda(), torch.from_numpy(starts).cuda(), b.scale,
             out=out)
        return out.float(), pkv.get_last_error()

    lens, starts = b.seq_lens.astype(np.int32), b.query_start_loc.astype(np.int32)
    good, flags = run(lens, starts)
    assert flags == 0
    first, last = slice(0, starts[1]), slice(starts[2], starts[3])
    width = meta["block_tables"].shape[1] * 16
    for value in (TOP, TOP - 7, TOP - 14, -2**31, -1, width + 1):
        L = lens.copy()
        L[1] = value
        out, flags = run(L, starts)
        assert flags == pkv.STATUS_BAD_QUERY, value
        for rows in (first, last):
            torch.testing.assert_close(out[rows], good[rows], rtol=2**-7, atol=1e-2)
        assert bool((out[starts[1]:starts[2]] == 7.0).all())
    for value in (TOP, -2**31):  # the end of the second sequence and the start of the third
        s = starts.copy()
        s[2] = value
        out, flags = run(lens, s)
        assert flags == pkv.STATUS_BAD_QUERY, value
        torch.testing.assert_close(out[first], good[first], rtol=2**-7, atol=1e-2)
        assert bool((out[starts[1]:] == 7.0).all())
