"""A page id outside the pool: its sequence's weights are not known, so its scores
stay as they were, whatever lies in other pages; the other sequences are right."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from test_weigh import SCALE, batch, call, cuda

pytestmark = pytest.mark.gpu

# sequences, rows of each, which of them is damaged: decode rows (also over many warps), drafts, a window, a
# prompt, few rows beside many
CASES = [([200, 90], [1, 1], 0), ([20000, 333], [1, 1], 0), ([130, 700, 64], [5, 8, 2], 1), ([200, 90], [60, 60], 0),
         ([640], [640], 0), ([700, 500, 33], [300, 1, 2], 0), ([700, 500, 33], [300, 1, 2], 1)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows,hurt", CASES)
@pytest.mark.parametrize("where", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("page", [-1, "behind", 2 ** 31 - 1])
def test_scores_of_a_damaged_sequence_stay(pkvlib, lens, rows, hurt, where, page, fp8):
    pkv.get_last_error()
    x = batch(lens, rows, 8, 2, seed=sum(lens), fp8=fp8, spare=2)
    NB = x["k"].shape[0]
    # page 0 belongs to no sequence here and holds no numbers
    free = np.setdiff1d(np.arange(NB), np.concatenate([x["tables"][b, :-(-n // 16)] for b, n in enumerate(x["lens"])]))[0]
    swap = np.arange(NB + 1)
    swap[[0, free]] = [free, 0]
    x["tables"] = swap[x["tables"]].astype(np.int32)
    for name in ("k", "scores") + (("ks",) if fp8 else ()):
        x[name] = x[name][swap[:NB]]
    pages = [x["tables"][b, :-(-n // 16)].copy() for b, n in enumerate(x["lens"])]
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, k_scale=x["ks"])
    d = cuda(x)
    d["block_tables"][hurt, int(where * (len(pages[hurt]) - 1))] = NB if page == "behind" else page
    for most in (max(rows), 0):
        d["scores"].copy_(torch.from_numpy(x["scores"]))
        got = call(x, d, max_query_len=most)
        assert pkv.get_last_error() == pkv.STATUS_BAD_BLOCK
        same = got.view(np.uint32) == x["scores"].view(np.uint32)
        for b in range(len(lens)):
            if b == hurt:
                assert same[pages[b]].all()
            else:
                on = bound[pages[b]] > 0
                assert (np.abs(got[pages[b]] - want[pages[b]])[on] <= bound[pages[b]][on]).all()
    # the next call, on sound tables, owes nothing to that one
    d["block_tables"].copy_(torch.from_numpy(x["tables"]))
    d["scores"].copy_(torch.from_numpy(x["scores"]))
    got = call(x, d, max_query_len=max(rows))
    assert pkv.get_last_error() == 0
    on = bound > 0
    assert (np.abs(got - want)[on] <= bound[on]).all()
