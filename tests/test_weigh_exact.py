"""Accumulated attention weights where scores are exact in fp32, so that nothing
but the exponentials and the sums can be off, and workspaces of exactly the size
asked for, with a guard on both sides."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from test_weigh import HEADS, SCALE, batch, call, cuda

pytestmark = pytest.mark.gpu


def bf16(a):
    return (np.asarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def whole_numbers(x, seed, q_step):
    """Queries of q_step times -8 to 8, keys of -4 to 4: every partial sum of a
    score is a whole number times q_step below 2^24, exact in any order."""
    rng = np.random.default_rng(seed)
    q = rng.integers(-8, 9, size=x["q"].shape) * q_step
    live = (x["q"] & 0x7FFF) != 0x7FC0
    x["q"] = np.where(live, bf16(q), x["q"])
    k = rng.integers(-4, 5, size=x["k"].shape)
    if x["fp8"]:
        code = {0: 0, 1: 0x38, 2: 0x40, 3: 0x44, 4: 0x48}  # E4M3
        codes = np.vectorize(code.get)(np.abs(k)).astype(np.uint8) | np.where(k < 0, 0x80, 0).astype(np.uint8)
        x["k"] = np.where((x["k"] & 0x7F) == 0x7F, x["k"], codes)
        x["ks"] = np.where(x["ks"] == 255, 255, 127).astype(np.uint8)
    else:
        x["k"] = np.where((x["k"] & 0x7FFF) == 0x7FC0, x["k"], bf16(k))
    return x


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows", [([400, 130, 77], [1, 1, 1]), ([700, 33, 200], [8, 3, 5]),
                                       ([300, 130], [100, 130]), ([1000, 40, 17], [300, 33, 1])])
@pytest.mark.parametrize("scale,q_step", [(2.0 ** -3, 1), (1.0, 1), (1.0, 16), (2.0, 64)])
def test_weights_of_exact_scores(pkvlib, lens, rows, scale, q_step, fp8):
    """Flat to sharply peaked rows (scores up to 2 * 64 * 128 * 32 = 2^19).  Each
    weight's exponent, its score less the row's log-sum N in powers of two, is off
    by two roundings at N's size (the maximum times the scale, the sum with the
    logarithm), the rounding of scale * log2(e), twice, and its own at the
    distance from the row's maximum, which is below 160 where the weight is not 0;
    a row's sum takes its maximum anew at most once a tile of 128 keys, off by
    two roundings at such a distance and exp2's 2^-21."""
    x = whole_numbers(batch(lens, rows, 8, 2, seed=sum(lens), fp8=fp8, pad=1), sum(rows), q_step)
    got = call(x, cuda(x), scale, decay=0.0)
    assert pkv.get_last_error() == 0
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], scale, 0.0, k_scale=x["ks"])
    biggest = scale * q_step * 8 * 4 * 128 / np.log(2.0)
    for b, L in enumerate(lens):
        tiles = -(-L // 128) + 1
        step = 2 * 160 * 2.0 ** -24 * np.log(2.0) + 2.0 ** -21
        rel = np.log(2.0) * (2 * 2.0 ** -24 * biggest + 3 * 160 * 2.0 ** -24) + tiles * step + 2.0 ** -20 \
            + (L + rows[b] * 4) * 2.0 ** -24
        rel *= 1.05  # second order
        pages = x["tables"][b, :-(-L // 16)]
        on = bound[pages] > 0
        w, g = want[pages][on], got[pages][on]
        assert (np.abs(g - w) <= rel * w + 1e-36).all()
        for h in range(2):
            live = np.arange(16 * len(pages)) < L
            total = got[pages, h].reshape(-1)[live].astype(np.float64).sum()
            assert abs(total - rows[b] * 4) <= rel * rows[b] * 4


def guarded(bytes_, fill=0xA5, guard=1 << 14):
    """(buffer, workspace): bytes_ between two guards."""
    whole = torch.full((bytes_ + 2 * guard,), fill, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    return whole, whole[guard:guard + bytes_], lambda: bool((whole[:guard] == fill).all()) and \
        bool((whole[guard + bytes_:] == fill).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(8))
def test_weigh_stays_within_its_workspace(pkvlib, seed, fp8):
    """Random batches, the bounds as tight as they can be, or unknown."""
    rng = np.random.default_rng(400 + seed)
    hq, hkv = HEADS[seed % len(HEADS)]
    B = int(rng.integers(1, 40))
    lens = np.exp(rng.uniform(0, np.log(1500), size=B)).astype(int)
    top = [1, 4, 9, 300][seed % 4]
    rows = np.minimum(lens, rng.integers(0, top + 1, size=B))
    if rows.sum() == 0:
        rows[0] = 1
    x = batch(lens, rows, hq, hkv, seed, fp8=fp8, pad=int(rng.integers(0, 3)))
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, k_scale=x["ks"])
    d = cuda(x)
    desc = pkv.make_desc(d["k_cache"], hq, x["tables"].shape[1])
    for most, keys in ((int(rows.max()), int((-(-x["lens"] // 16)).sum()) * 16), (0, 0)):
        size = pkv.workspace_size_weigh(desc, B, x["q"].shape[0], max_query_len=most, num_keys=keys)
        _, ws, whole = guarded(size)
        d["scores"].copy_(torch.from_numpy(x["scores"]))
        got = call(x, d, workspace=ws, max_query_len=most, num_keys=keys)
        assert pkv.get_last_error() == 0 and whole()
        on = bound > 0
        assert (np.abs(got - want)[on] <= bound[on]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("keys", [0, 16, 304, 640, 1200])
def test_weigh_keys_that_no_bound_holds(pkvlib, rows, keys, fp8):
    """Sequences that share a prefix hold more tokens than the pool has, or than
    num_keys says: each is right, or left alone and the call flagged, and
    nothing is written behind the workspace."""
    pkv.get_last_error()
    x = batch([300, 290, 310, 260, 300, 281], [rows] * 6, 8, 2, seed=22, fp8=fp8)
    own = np.unique(np.concatenate([x["tables"][0, :19]] + [x["tables"][b, 15:-(-x["lens"][b] // 16)] for b in range(6)]))
    x["tables"][1:, :15] = x["tables"][0, :15]
    renumber = np.full(x["k"].shape[0] + 1, len(own), np.int32)
    renumber[own] = np.arange(len(own))
    x["tables"] = renumber[x["tables"]]
    for name in ("k", "scores") + (("ks",) if fp8 else ()):
        x[name] = x[name][own]
    first = [240] * 6
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, first=first,
                          k_scale=x["ks"])
    d = cuda(x)
    desc = pkv.make_desc(d["k_cache"], 8, x["tables"].shape[1])
    size = pkv.workspace_size_weigh(desc, 6, x["q"].shape[0], max_query_len=rows, num_keys=keys)
    _, ws, whole = guarded(size)
    got = call(x, d, first=torch.full((6,), 240, dtype=torch.int32, device="cuda"), workspace=ws, max_query_len=rows,
               num_keys=keys)
    flags = pkv.get_last_error()
    assert whole()
    right = []
    for b in range(6):
        pages = x["tables"][b, 15:-(-x["lens"][b] // 16)]
        on = bound[pages] > 0
        same = np.array_equal(got[pages].view(np.uint32), x["scores"][pages].view(np.uint32))
        ok = bool((np.abs(got[pages] - want[pages])[on] <= bound[pages][on]).all())
        assert ok != same
        right.append(ok)
    shared = x["tables"][0, :15]
    assert np.array_equal(got[shared].view(np.uint32), x["scores"][shared].view(np.uint32))
    assert right == sorted(right, reverse=True)  # the first that does not fit ends the list
    assert flags == (0 if all(right) else pkv.STATUS_BAD_QUERY)
    if rows <= 4:  # scores are kept for as many keys as the bound says, 608 where it is the pool's tokens
        fits = int(np.searchsorted(np.cumsum(-(-x["lens"] // 16) * 16), keys or len(own) * 16, side="right"))
        assert sum(right) == fits < 6
