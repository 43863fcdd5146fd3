"""The first evictions of a process, from several host threads at once: what the
library asks the device once (cluster sizes, shared memory) is asked by one of
them and read by all."""

import ctypes
import shutil
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from test_evict import batch

pytestmark = pytest.mark.gpu

THREADS = 12


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hkv", [([9000, 1200], 2), ([400, 90, 333], 1)])
def test_first_evictions_of_several_threads(pkvlib, tmp_path, lens, hkv, fp8):
    """Each thread on its own stream, pools and workspace; a copy of the library
    has asked nothing yet."""
    copy = shutil.copy(pkv.library_path, tmp_path / "libpkv_copy.so")
    lib = pkv.open_library(str(copy))
    x = batch(lens, hkv, seed=sum(lens), fp8=fp8, kind="ties")
    keep = [n // 2 for n in lens]
    B, M = x["tables"].shape
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    dev = lambda p: torch.from_numpy(p.view(np.int16) if p.dtype == np.uint16 else p).cuda()
    tables, seq_lens, d_keep = i32(x["tables"]), i32(x["lens"]), i32(keep)
    state = [[dev(p) for p in x["pools"]] + [torch.from_numpy(x["scores"]).cuda()] for _ in range(THREADS)]
    new = torch.zeros(THREADS, B, dtype=torch.int32, device="cuda")
    desc = pkv.Desc(x["scores"].shape[0], 16, hkv, hkv, 128, M)
    size = ctypes.c_size_t(0)
    assert lib.pkv_evict_workspace_size(ctypes.byref(desc), B, ctypes.byref(size)) == 0
    ws = [torch.empty(size.value, dtype=torch.uint8, device="cuda") for _ in range(THREADS)]
    streams = [torch.cuda.Stream() for _ in range(THREADS)]
    torch.cuda.synchronize()
    start, rc = threading.Barrier(THREADS), [None] * THREADS
    p = lambda t: ctypes.c_void_p(t.data_ptr())

    def call(i):
        torch.cuda.set_device(0)
        fn = lib.pkv_evict_fp8 if fp8 else lib.pkv_evict
        args = [*map(p, state[i]), p(tables), p(seq_lens), p(d_keep), None, 3, B, p(new[i]), p(ws[i]), size.value,
                ctypes.byref(desc), ctypes.c_void_p(streams[i].cuda_stream)]
        start.wait()
        rc[i] = fn(*args)

    threads = [threading.Thread(target=call, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert rc == [0] * THREADS
    pools, scores, le = E.evict(x["pools"], x["scores"], x["tables"], x["lens"], keep, None, 3)
    for i in range(THREADS):
        assert new[i].tolist() == le.tolist()
        assert np.array_equal(state[i][-1].cpu().numpy(), scores)
        for got, want in zip(state[i], pools):
            assert np.array_equal(got.cpu().numpy().view(want.dtype), want)
