"""Bounded waits of the latent attention kernels: in a test build whose first
query copy is announced but never made, every wait behind it runs out; the
kernels flag PKV_STATUS_TIMEOUT, let what is under way land, free their TMEM and
return, and the device stays usable.  No wait is unbounded."""

import ctypes

import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from test_latent import WIDE, Case
from test_timeout import _flags, _p, _stream, dropped_copy_lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,width", [(16, 1), (64, 1), (128, WIDE)])
def test_missing_queries_time_out_and_leave_the_device_usable(pkvlib, dropped_copy_lib, H, width):  # noqa: F811
    lib = dropped_copy_lib
    c = Case([700, 33, 130], [1, 1, 2], H, seed=1, width=width)
    q, pool, tables, lens, qsl, scale = c.args()
    out = torch.zeros(c.q.shape[0], H, 512, device="cuda", dtype=torch.bfloat16)
    desc = pkv.make_latent_desc(pool, H, tables.shape[1])
    size = ctypes.c_size_t(0)
    assert lib.pkv_attend_latent_workspace_size(ctypes.byref(desc), 3, c.q.shape[0], ctypes.byref(size)) == 0
    ws = torch.zeros(size.value, device="cuda", dtype=torch.uint8)
    assert _flags(lib) == 0
    for _ in range(2):
        assert lib.pkv_attend_latent(_p(q), _p(pool), _p(tables), _p(lens), _p(qsl), 3, c.q.shape[0], 2, scale, _p(out),
                                     _p(ws), ws.numel(), ctypes.byref(desc), _stream()) == 0
        assert _flags(lib) & pkv.STATUS_TIMEOUT
    c.check(pkv.attend_latent(*c.args(), max_query_len=2))
    assert pkv.get_last_error() == 0
