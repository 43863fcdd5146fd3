"""attend_latent where the batch has more tiles of rows than there are CTAs (or
pairs of them): equal shares of the work, several pieces a share, tiles cut
among shares.  Against float64 within the bound that
oracle.rotary_latent.attend_latent derives, and bit for bit from call to call
while another stream keeps the memory busy."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from test_latent import SCALE, WIDE, Case

pytestmark = pytest.mark.gpu


def lengths(seed, n, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi, size=n, endpoint=True)


def rising(c, step=0.25):
    """Keys that score higher and higher along each sequence."""
    u = torch.randn(576, device="cuda")
    u /= u.norm()
    c.q[:] = (u * 30).to(torch.bfloat16)
    for b, L in enumerate(c.lens):
        j = np.arange(int(L))
        page, row = (torch.from_numpy(a).cuda().long() for a in (c.tables[b, j // 16], j % 16))
        c.pool[page, row] += (step * torch.from_numpy(j).cuda()[:, None] * u).to(torch.bfloat16)


def check_repeatedly(c, times=40, **kw):
    """Every call the same bits, the first within the bound; meanwhile copies on
    another stream take the memory, and the instructions out of the caches, so
    that single warps fall behind by microseconds."""
    pkv.get_last_error()
    args = c.args()
    ws = torch.empty(pkv.workspace_size_latent(pkv.make_latent_desc(c.pool, c.H, c.tables.shape[1]), len(c.lens),
                                               c.q.shape[0]), dtype=torch.uint8, device="cuda")
    noise = torch.empty(2, 1 << 26, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    first = pkv.attend_latent(*args, workspace=ws, **kw)
    c.check(first)
    for i in range(0, times, 20):
        outs = []
        for _ in range(min(20, times - i)):
            with torch.cuda.stream(side):
                noise[0].copy_(noise[1])
            outs.append(pkv.attend_latent(*args, workspace=ws, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(first.view(torch.int16), o.view(torch.int16)) for o in outs)
    assert pkv.get_last_error() == 0


def test_whole_tiles_of_one_step_follow_each_other_on_pairs(pkvlib):
    """Prompts of at most 128 tokens and 128 heads: every tile is one token and
    one step over the keys, a pair has nine or so, and each ends with an
    exchange of row sums."""
    lens = [128, 100, 77, 128, 5, 90, 128, 1]
    check_repeatedly(Case(lens, lens, 128, seed=21, width=WIDE), max_query_len=128)


@pytest.mark.parametrize("H", [65, 96, 128])
def test_equal_shares_on_pairs(pkvlib, H):
    lens = lengths(22 + H, 90, 1, 300)
    check_repeatedly(Case(lens, np.ones(90, int), H, seed=22, width=WIDE), max_query_len=1)


def test_tiles_cut_among_several_pairs(pkvlib):
    lens = np.concatenate([lengths(23, 50, 1, 200), [6000, 2049], lengths(24, 50, 1, 200), [3000]])
    q_lens = np.ones(len(lens), int)
    q_lens[[50, 102]] = 3
    check_repeatedly(Case(lens, q_lens, 96, seed=23), times=10, max_query_len=3)


@pytest.mark.parametrize("H,most", [(96, 1), (40, 3)])
def test_a_second_round_over_several_pieces_on_pairs(pkvlib, H, most):
    """Scores that leave the first reference far behind: pairs go through their
    shares again, several pieces each, whole ones and cut ones."""
    lens = lengths(25, 90, most, 300)
    c = Case(lens, 1 + np.arange(90) % most, H, seed=25, width=WIDE)
    rising(c)
    check_repeatedly(c, times=10)


@pytest.mark.parametrize("H", [16, 20, 40, 64])
def test_equal_shares_on_single_ctas(pkvlib, H):
    """Most sequences' last tile has pages that are not loaded; what is written
    over them must not come before the tile two before is done with them."""
    lens = lengths(26 + H, 170, 1, 300)
    check_repeatedly(Case(lens, np.ones(170, int), H, seed=26), times=500, max_query_len=1)


def test_whole_tiles_follow_each_other_on_single_ctas(pkvlib):
    """Prompts whose tiles of 64 rows are one to four steps long, a dozen whole
    ones a CTA: each begins with new references where the one before ended with
    its row sums."""
    lens = [250, 64, 100, 130, 192, 7]
    check_repeatedly(Case(lens, lens, 128, seed=27), max_query_len=250)


@pytest.mark.parametrize("H", [12, 64])
def test_tiles_cut_among_several_ctas(pkvlib, H):
    lens = np.concatenate([lengths(28, 90, 1, 200), [9000, 2049], lengths(29, 70, 1, 200), [4096]])
    check_repeatedly(Case(lens, np.ones(len(lens), int), H, seed=28), times=10, max_query_len=1)


@pytest.mark.parametrize("H", [16, 64])
def test_references_raised_over_several_pieces_on_single_ctas(pkvlib, H):
    lens = lengths(30, 170, 1, 300)
    c = Case(lens, np.ones(170, int), H, seed=30)
    rising(c)
    check_repeatedly(c, times=10, max_query_len=1)


def test_more_sequences_than_a_warp_of_the_plan_scans_at_once(pkvlib):
    """As many sequences as a call takes, some without rows, some without
    tokens."""
    lens = lengths(31, 2048, 0, 40)
    q_lens = np.minimum(lens, lengths(32, 2048, 0, 1))
    check_repeatedly(Case(lens, q_lens, 8, seed=31), times=5, max_query_len=1)
    check_repeatedly(Case(lens, q_lens, 72, seed=31, width=WIDE), times=5, max_query_len=1)


@pytest.mark.parametrize("H,width", [(20, 1), (40, 1), (70, 1), (70, WIDE), (96, WIDE)])
def test_a_row_goes_by_its_own_tile_alone(pkvlib, H, width):
    """A tile's copy of queries runs on into the next sequence's, or into tokens
    behind the last one: whatever these hold, a sequence's bits stay the same."""
    pkv.get_last_error()
    c = Case([300, 900, 77], [1, 1, 1], H, seed=33, extra_tokens=4, width=width)
    want = pkv.attend_latent(*c.args(), max_query_len=1)
    c.check(want)
    q0 = c.q.clone()
    for value in (3e4, -3e4, 3e38, float("inf"), float("nan")):
        for tokens in ([1], [2], [3, 4, 5, 6]):
            c.q.copy_(q0)
            c.q[tokens] *= value
            got = pkv.attend_latent(*c.args(), max_query_len=1)
            others = [b for b in range(3) if b not in tokens]
            same = torch.equal(got[others].view(torch.int16), want[others].view(torch.int16))
            assert same, (value, tokens)
    assert pkv.get_last_error() == 0
