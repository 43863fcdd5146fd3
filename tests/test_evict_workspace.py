"""Eviction in workspaces of exactly the size asked for, between guards, whatever
they held: the list of kept tokens is all that is read there.  (The fills are
tokens of the sequences, so that a list entry that was not written would move a
wrong row and not reach out of bounds.)"""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from test_evict import batch, check
from test_weigh_exact import guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("fill", [0, 1])
@pytest.mark.parametrize("lens,hkv,width,kind", [
    ([500, 33, 17, 257], 2, None, "ties"),                    # a CTA an item
    ([5000, 4097, 20], 2, None, "ties"),                      # clusters
    ([60, 300, 45], 2, 700, "any"),                           # short sequences in wide tables
    (list(range(16, 400, 2)), 2, None, "weights"),            # items fill the GPU
])
def test_evict_stays_within_its_workspace(pkvlib, lens, hkv, width, kind, fill, fp8):
    x = batch(lens, hkv, seed=sum(lens), fp8=fp8, width=width, kind=kind)
    desc = pkv.Desc(x["scores"].shape[0], 16, hkv, hkv, 128, x["tables"].shape[1])
    size = pkv.workspace_size_evict(desc, len(lens))
    _, ws, whole = guarded(size)
    ws.view(torch.int32).fill_(fill)
    check(x, [n // 2 for n in lens], [n // 9 for n in lens], 5, workspace=ws)
    assert whole()
    # keep one token, all but one, and none
    for keep in ([1] * len(lens), [n - 1 for n in lens], [0] * len(lens)):
        ws.view(torch.int32).fill_(fill)
        check(x, keep, None, 0, workspace=ws)
        assert whole()
    assert np.array_equal(x["lens"], lens)
