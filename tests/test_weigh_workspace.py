"""What a workspace held before a call does not matter: every kernel of
accumulated attention weights reads there only what the call has written."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from test_weigh import SCALE, batch, cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [1, 2, 3, 4, 5, 6, 7, 8, 40])
@pytest.mark.parametrize("word", [0x7F800000, 0xFF800000, 0x7FC00000, 0x7F7FFFFF, 0xFF7FFFFF, 0x00000000, 0x3F800000],
                         ids=["inf", "-inf", "nan", "max", "min", "zero", "one"])
def test_any_workspace(pkvlib, word, most, fp8):
    """Every number of row tiles and score quads, fewer rows beside the most."""
    lens, rows = [300, most + 30, 70, 17], [most, 1, max(1, most - 1), 2 if most > 1 else 1]
    x = batch(lens, rows, 8, 2, seed=most, fp8=fp8, pad=1)
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, 0.5, k_scale=x["ks"])
    d = cuda(x)
    desc = pkv.make_desc(d["k_cache"], 8, x["tables"].shape[1])
    size = pkv.workspace_size_weigh(desc, len(lens), x["q"].shape[0], max_query_len=most)
    words = torch.from_numpy(np.full(-(-size // 4), word, np.uint32).view(np.int32)).cuda()
    ws = words.view(torch.uint8)
    (pkv.weigh_fp8 if fp8 else pkv.weigh)(scale=SCALE, decay=0.5, workspace=ws, max_query_len=most, **d)
    assert pkv.get_last_error() == 0
    got = d["scores"].cpu().numpy()
    on = bound > 0
    assert np.isfinite(got[on]).all() and (np.abs(got - want)[on] <= bound[on]).all()
    assert np.array_equal(got[~on].view(np.uint32), x["scores"][~on].view(np.uint32))
