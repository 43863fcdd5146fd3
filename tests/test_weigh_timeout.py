"""Bounded waits of the tensor-core kernels of accumulated attention weights: in a
test build whose first pair of tiles of every CTA is announced but never copied,
every wait behind it runs out in both passes.  The kernels flag
PKV_STATUS_TIMEOUT, let what is under way land, free their TMEM and return; the
kernels that join pieces read nothing but what this call has written, in a
workspace full of numbers that are no items, and the device stays usable.  No
wait is unbounded."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from test_timeout import _flags, _p, _stream, dropped_copy_lib  # noqa: F401
from test_weigh import SCALE, batch, call, compare, cuda

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows,hq", [([700, 350, 16, 70], [250, 350, 16, 1], 8), ([1100], [1100], 2),
                                          ([45] * 200 + [3000, 9], [33] * 200 + [64, 2], 8)])
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_waits_that_run_out_leave_no_item_unwritten(pkvlib, dropped_copy_lib, lens, rows, hq, fp8, fill):  # noqa: F811
    lib = dropped_copy_lib
    x = batch(lens, rows, hq, 2, seed=sum(lens), fp8=fp8, pad=1)
    d = cuda(x)
    B, T, M = len(lens), x["q"].shape[0], x["tables"].shape[1]
    desc = pkv.make_desc(d["k_cache"], hq, M)
    size = ctypes.c_size_t(0)
    assert lib.pkv_weigh_workspace_size(ctypes.byref(desc), B, T, 0, 0, ctypes.byref(size)) == 0
    ws = torch.full((size.value + GUARD,), fill, device="cuda", dtype=torch.uint8)
    pools = [_p(d["k_cache"])] + ([_p(d["k_scale"])] if fp8 else [])
    fn = lib.pkv_weigh_fp8 if fp8 else lib.pkv_weigh
    assert _flags(lib) == 0
    for _ in range(2):
        d["scores"].copy_(torch.from_numpy(x["scores"]))
        ws.fill_(fill)
        assert fn(_p(d["q"]), *pools, _p(d["scores"]), _p(d["block_tables"]), _p(d["seq_lens"]),
                  _p(d["query_start_loc"]), None, None, B, T, 0, 0, SCALE, 1.0, _p(ws), size.value, ctypes.byref(desc),
                  _stream()) == 0
        assert _flags(lib) == pkv.STATUS_TIMEOUT
        assert (ws[size.value:] == fill).all()
        got = d["scores"].cpu().numpy()
        # every CTA lost its first pair: no weight of many rows is a number, those of few rows are right
        few = np.flatnonzero(np.asarray(rows) * hq // 2 <= 32)
        want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, k_scale=x["ks"])
        touched = bound > 0
        right = np.zeros(touched.shape[0], bool)
        for b in few:
            right[x["tables"][b, :-(-x["lens"][b] // 16)]] = True
        assert np.isnan(got[touched & ~right[:, None, None]]).all()
        on = touched & right[:, None, None]
        assert (np.abs(got - want)[on] <= bound[on]).all()
        assert np.array_equal(got[~touched].view(np.uint32), x["scores"][~touched].view(np.uint32))
    d["scores"].copy_(torch.from_numpy(x["scores"]))
    compare(x, call(x, d))
    assert pkv.get_last_error() == 0
