"""Accumulated attention weights against the float64 form, within a bound that
is derived element by element (oracle/eviction.py)."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E
from oracle.pkv_oracle import bf16_to_f64

gpu = pytest.mark.gpu
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
NULL, ALIGN, SHAPE, RANGE, WORKSPACE = -1, -2, -3, -4, -5
SCALE = 128 ** -0.5


# ---- host -----------------------------------------------------------------------


def test_weights_by_hand():
    """Two rows of two heads over three keys, each weight from its formula."""
    rng = np.random.default_rng(0)
    bf = lambda a: (np.asarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    q, k = bf(rng.standard_normal((2, 2, 128))), bf(rng.standard_normal((2, 1, 16, 128)))
    scores = np.full((2, 1, 16), 10.0, np.float32)
    out, bound = E.weigh(q, k, scores, [[1]], [3], [0, 2], 0.1, decay=0.5)
    w = np.zeros(3)
    for j in range(2):
        for h in range(2):
            s = [0.1 * float(bf16_to_f64(q)[j, h] @ bf16_to_f64(k)[1, 0, i]) for i in range(2 + j)]
            for i in range(2 + j):
                w[i] += np.exp(s[i]) / sum(np.exp(x) for x in s)
    assert np.allclose(out[1, 0, :3], w + [5.0, 0.0, 0.0], rtol=1e-12) and abs(w.sum() - 4) < 1e-12
    assert (out[0] == 10).all() and (out[1, 0, 3:] == 10).all() and (bound[1, 0, 3:] == 0).all()
    kept, _ = E.weigh(q, k, scores, [[1]], [3], [0, 2], 0.1, decay=0.0, first=[2], scored=[3])
    assert (kept[1, 0, :2] == 10).all() and abs(kept[1, 0, 2] - w[2]) < 1e-12


def _weigh(lib, fp8=False, desc=None, B=4, T=4, most=0, keys=0, scale=0.1, decay=1.0, bytes_=1 << 20, **ptr):
    p = dict(q=FAKE, kc=FAKE, ks=FAKE, scores=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, first=FAKE, scored=FAKE, ws=FAKE)
    p.update(ptr)
    d = desc or pkv.Desc(64, 16, 2, 8, 128, 16)
    pools = [p["kc"], p["ks"]] if fp8 else [p["kc"]]
    fn = lib.pkv_weigh_fp8 if fp8 else lib.pkv_weigh
    return fn(p["q"], *pools, p["scores"], p["bt"], p["sl"], p["qsl"], p["first"], p["scored"], B, T, most, keys, scale,
              decay, p["ws"], bytes_, ctypes.byref(d), None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), RANGE), (dict(B=2049), RANGE), (dict(T=-1), RANGE), (dict(T=2 ** 31 - 1), RANGE),
    (dict(scale=-0.1), RANGE), (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE),
    (dict(decay=-1.0), RANGE), (dict(decay=float("nan")), RANGE), (dict(decay=float("inf")), RANGE),
    (dict(q=None), NULL), (dict(kc=None), NULL), (dict(scores=None), NULL), (dict(bt=None), NULL), (dict(sl=None), NULL),
    (dict(qsl=None), NULL), (dict(ws=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(kc=FAKE + 8), ALIGN),
    (dict(scores=FAKE + 4), ALIGN), (dict(ws=FAKE + 128), ALIGN), (dict(first=FAKE + 2), ALIGN),
    (dict(scored=FAKE + 2), ALIGN), (dict(desc=pkv.Desc(64, 16, 2, 8, 64, 16)), SHAPE),
    (dict(desc=pkv.Desc(64, 16, 2, 12, 128, 16)), SHAPE), (dict(desc=pkv.Desc(64, 16, 2, 8, 128, 1 << 27)), RANGE),
    (dict(desc=pkv.Desc(1 << 26, 16, 2, 8, 128, 16)), RANGE),
])
def test_weigh_refuses(pkvlib, fp8, bad, code):
    before = pkvlib.pkv_launch_count()
    assert _weigh(pkvlib, fp8=fp8, **bad) == code
    assert _weigh(pkvlib, fp8=fp8, B=0) == 0 and _weigh(pkvlib, fp8=fp8, T=0) == 0
    assert pkvlib.pkv_launch_count() == before


def test_weigh_workspace_size_refuses(pkvlib):
    n = ctypes.c_size_t(0)
    d = ctypes.byref(pkv.Desc(64, 16, 2, 8, 128, 16))
    for B, T in ((-1, 4), (2049, 4), (4, -1)):
        assert pkvlib.pkv_weigh_workspace_size(d, B, T, 0, 0, ctypes.byref(n)) == RANGE
    assert pkvlib.pkv_weigh_workspace_size(d, 4, 4, 0, 0, None) == NULL
    assert pkvlib.pkv_weigh_workspace_size(None, 4, 4, 0, 0, ctypes.byref(n)) == NULL


# ---- GPU ------------------------------------------------------------------------


def batch(lens, rows, hq, hkv, seed, fp8=False, width=None, pad=0, peak=1.0, spare=3):
    """A batch on the host and on the device.  What nothing may use is NaN:
    cached rows past a sequence's end, scores of tokens without one, query
    rows behind the last sequence."""
    rng = np.random.default_rng(seed)
    lens, rows = np.asarray(lens, np.int32), np.asarray(rows, np.int32)
    need = -(-lens // 16)
    NB = int(need.sum()) + spare
    M = width or max(1, int(need.max()))
    tables = np.full((len(lens), M), NB, np.int32)
    perm, at = rng.permutation(NB), 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    qsl = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(qsl[-1]) + pad
    bf = lambda a: (np.asarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    q = bf(rng.standard_normal((T, hq, 128)) * peak)
    q[qsl[-1]:] = 0x7FC0
    shape = (NB, hkv, 16)
    used = np.zeros((NB, 16), bool)
    for b, L in enumerate(lens):
        j = np.arange(L)
        used[tables[b, j // 16], j % 16] = True
    x = dict(lens=lens, rows=rows, qsl=qsl, tables=tables, q=q, fp8=fp8)
    x["scores"] = rng.random(shape).astype(np.float32)
    x["scores"].transpose(0, 2, 1)[~used] = np.nan
    if fp8:
        x["k"] = rng.integers(0, 256, size=shape + (128,), dtype=np.uint8)
        x["k"][(x["k"] & 0x7F) == 0x7F] = 0x33
        x["ks"] = rng.integers(117, 121, size=shape, dtype=np.uint8)
        x["k"].transpose(0, 2, 1, 3)[~used] = 0x7F
        x["ks"].transpose(0, 2, 1)[~used] = 255
    else:
        x["k"] = bf(rng.standard_normal(shape + (128,)))
        x["k"].transpose(0, 2, 1, 3)[~used] = 0x7FC0
        x["ks"] = None
    return x


def cuda(x):
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    bf = lambda a: torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    d = dict(q=bf(x["q"]), scores=torch.from_numpy(x["scores"].copy()).cuda(), block_tables=i32(x["tables"]),
             seq_lens=i32(x["lens"]), query_start_loc=i32(x["qsl"]),
             k_cache=torch.from_numpy(x["k"]).cuda() if x["fp8"] else bf(x["k"]))
    if x["fp8"]:
        d["k_scale"] = torch.from_numpy(x["ks"]).cuda()
    return d


def call(x, d, scale=SCALE, **kw):
    (pkv.weigh_fp8 if x["fp8"] else pkv.weigh)(scale=scale, **d, **kw)
    return d["scores"].cpu().numpy()


def compare(x, got, scale=SCALE, decay=1.0, first=None, scored=None):
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], scale, decay, first, scored,
                          k_scale=x["ks"])
    touched = bound > 0
    assert np.array_equal(got[~touched].view(np.uint32), x["scores"][~touched].view(np.uint32))
    assert np.isfinite(got[touched]).all()
    over = np.abs(got[touched] - want[touched]) / bound[touched]
    assert over.size == 0 or over.max() <= 1.0, f"{over.max():.2f} of the bound"


def check(x, scale=SCALE, decay=1.0, first=None, scored=None, flags=0, **kw):
    i32 = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).cuda()
    d = cuda(x)
    got = call(x, d, scale, decay=decay, first=i32(first), scored=i32(scored), **kw)
    assert pkv.get_last_error() == flags
    compare(x, got, scale, decay, first, scored)
    return got


HEADS = [(1, 1), (8, 2), (4, 1), (8, 1), (16, 1), (16, 8)]


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens", [[1], [17, 5, 16, 240], [300, 1, 33, 128, 129, 127, 64]])
def test_weigh_decode_rows(pkvlib, lens, hq, hkv, fp8):
    x = batch(lens, [1] * len(lens), hq, hkv, seed=sum(lens) + hq, fp8=fp8, pad=2)
    check(x, max_query_len=1)
    check(x, decay=0.75)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (16, 1)])
@pytest.mark.parametrize("lens,rows", [([9, 200, 40], [2, 5, 0]), ([64, 300, 8, 100], [8, 1, 8, 3]),
                                       ([500, 40, 130], [9, 33, 1]), ([257, 400], [129, 64]),
                                       ([700, 350, 16, 70], [250, 350, 16, 1]), ([1100], [1100])])
def test_weigh_chunks(pkvlib, lens, rows, hq, hkv, fp8):
    """Drafts, windows, chunks over a context, whole prompts, sequences without rows."""
    x = batch(lens, rows, hq, hkv, seed=sum(lens) + hq, fp8=fp8, pad=3)
    check(x, max_query_len=max(rows))
    check(x, decay=0.0)


@gpu
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65])
def test_weigh_row_counts(pkvlib, n):
    """Both sides of every choice of kernel and tile by the number of rows."""
    x = batch([n, n + 200, 600], [n, n, n], 8, 2, seed=n)
    check(x, max_query_len=n)
    check(x, decay=0.5)


@gpu
@pytest.mark.parametrize("n", [2, 3, 4, 5, 6, 7, 8, 9])
def test_weigh_row_counts_fp8(pkvlib, n):
    """Every number of MMA tiles of rows on E4M3 pages, fewer rows beside the most."""
    x = batch([n + 700, n, 350, 17], [n, n, 1, 2], 8, 2, seed=50 + n, fp8=True)
    check(x, max_query_len=n)
    check(x, decay=0.5)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_weigh_scores_kept_and_new(pkvlib, fp8):
    """first: no score is written; scored: what is held from there on is not
    read (NaN here); decay 0 reads none at all."""
    x = batch([150, 90, 300], [1, 2, 50], 8, 2, seed=3, fp8=fp8)
    first, scored = [20, 0, 999], [100, 90, 0]
    check(x, decay=0.9, first=first, scored=scored)
    for b in range(3):
        j = np.arange(scored[b], x["lens"][b])
        x["scores"][x["tables"][b, j // 16], :, j % 16] = np.nan
    check(x, decay=0.9, first=[0, 0, 0], scored=scored)
    for b in range(3):
        j = np.arange(x["lens"][b])
        x["scores"][x["tables"][b, j // 16], :, j % 16] = np.inf
    check(x, decay=0.0, first=first, scored=[-5, 2 ** 31 - 1, 40])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("peak,scale", [(30.0, SCALE), (1.0, 0.0), (1e-30, SCALE), (300.0, 1.0)])
def test_weigh_peaked_and_flat(pkvlib, peak, scale, fp8):
    """One key takes nearly all of a row's weight; all keys the same."""
    x = batch([400, 130, 77], [1, 100, 3], 8, 2, seed=4, fp8=fp8, peak=peak)
    check(x, scale=scale, decay=0.0)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_weigh_long_and_ragged(pkvlib, fp8):
    """A sequence split among many warps beside short ones and one of chunked rows."""
    x = batch([20000, 3, 700, 16], [1, 1, 40, 2], 8, 2, seed=5, fp8=fp8, width=2000)
    check(x, decay=1.0)


@gpu
def test_weigh_many_sequences(pkvlib):
    rng = np.random.default_rng(6)
    lens = rng.integers(1, 60, size=300)
    x = batch(lens, np.minimum(lens, rng.integers(0, 4, size=300)), 4, 2, seed=6)
    check(x, max_query_len=3, num_keys=int((-(-lens // 16)).sum()) * 16)


@gpu
@pytest.mark.parametrize("seed", range(6))
def test_weigh_random(pkvlib, seed):
    rng = np.random.default_rng(100 + seed)
    hq, hkv = HEADS[rng.integers(len(HEADS))]
    B = int(rng.integers(1, 12))
    lens = np.exp(rng.uniform(0, np.log(2500), size=B)).astype(int)
    rows = np.minimum(lens, np.exp(rng.uniform(-0.7, np.log(300), size=B)).astype(int))
    x = batch(lens, rows, hq, hkv, seed, fp8=bool(seed % 2), pad=int(rng.integers(0, 3)))
    check(x, decay=float(rng.choice([0.0, 0.9, 1.0])), first=rng.integers(0, 30, size=B),
          max_query_len=int(rng.choice([0, max(1, rows.max())])))


@gpu
def test_weigh_same_bits(pkvlib):
    x = batch([900, 60, 2000], [200, 1, 5], 8, 2, seed=7)
    first = call(x, cuda(x))
    for _ in range(5):
        assert np.array_equal(call(x, cuda(x)).view(np.uint32), first.view(np.uint32))


@gpu
def test_weigh_bounds_that_do_not_hold_are_flagged(pkvlib):
    pkv.get_last_error()
    x = batch([64, 100, 30], [1, 20, 2], 8, 2, seed=8)
    got = call(x, cuda(x), max_query_len=2)  # the second has more rows
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, k_scale=None)
    second = np.zeros(x["scores"].shape[0], bool)
    second[x["tables"][1, :7]] = True
    touched = (bound > 0) & ~second[:, None, None]
    assert (np.abs(got - want)[touched] <= bound[touched]).all()
    assert np.array_equal(got[second].view(np.uint32), x["scores"][second].view(np.uint32))


@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_weigh_keys_beyond_the_bound_are_flagged(pkvlib, rows):
    """num_keys too small by far: what fits is right, the rest is left alone."""
    pkv.get_last_error()
    x = batch([600, 500, 700, 400], [rows] * 4, 8, 2, seed=20)
    got = call(x, cuda(x), num_keys=608, max_query_len=rows)
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE)
    done = []
    for b in range(4):
        pages = x["tables"][b, :-(-x["lens"][b] // 16)]
        same = np.array_equal(got[pages].view(np.uint32), x["scores"][pages].view(np.uint32))
        touched = bound[pages] > 0
        right = (np.abs(got[pages] - want[pages])[touched] <= bound[pages][touched]).all()
        assert same or right
        done.append(bool(right))
    assert done[0] and not done[3]


@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_weigh_sequences_on_a_shared_prefix(pkvlib, rows):
    """Six sequences share 15 pages, their first tokens: together more tokens
    than the pool has, which num_keys says."""
    pkv.get_last_error()
    x = batch([300, 290, 310, 260, 300, 281], [rows] * 6, 8, 2, seed=22)
    own = np.unique(np.concatenate([x["tables"][0, :19]] + [x["tables"][b, 15:-(-x["lens"][b] // 16)] for b in range(6)]))
    x["tables"][1:, :15] = x["tables"][0, :15]
    renumber = np.full(x["k"].shape[0] + 1, len(own), np.int32)
    renumber[own] = np.arange(len(own))
    x["tables"] = renumber[x["tables"]]
    x["k"], x["scores"] = x["k"][own], x["scores"][own]
    keys = int((-(-x["lens"] // 16)).sum()) * 16
    assert keys > x["k"].shape[0] * 16
    check(x, first=[240] * 6, num_keys=keys, max_query_len=rows)
    d = cuda(x)
    call(x, d, first=torch.full((6,), 240, dtype=torch.int32, device="cuda"), max_query_len=rows)
    assert pkv.get_last_error() in (0, pkv.STATUS_BAD_QUERY)  # the pool's tokens do not bound them


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_weigh_most_sequences(pkvlib, fp8):
    """As many sequences as a call takes, a few with a window of rows."""
    rng = np.random.default_rng(23)
    lens = rng.integers(1, 40, size=2048)
    rows = np.where(rng.random(2048) < 0.02, np.minimum(lens, 30), np.minimum(lens, rng.integers(0, 3, size=2048)))
    x = batch(lens, rows, 4, 1, seed=23, fp8=fp8)
    check(x, decay=0.5)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_weigh_fewer_rows_than_a_capture_had(pkvlib, fp8):
    """Captured where every sequence has the most rows (no kernels of few rows),
    replayed with few rows, none, and padding behind the last sequence."""
    x = batch([300, 64, 200], [40, 40, 40], 8, 2, seed=21, fp8=fp8)
    d = cuda(x)
    (pkv.weigh_fp8 if fp8 else pkv.weigh)(scale=SCALE, max_query_len=40, **cuda(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (pkv.weigh_fp8 if fp8 else pkv.weigh)(scale=SCALE, max_query_len=40, **d)
    graph.replay()
    torch.cuda.synchronize()
    compare(x, d["scores"].cpu().numpy())
    qsl = np.array([0, 1, 1, 38], np.int32)
    y = dict(x, qsl=qsl, scores=d["scores"].cpu().numpy())
    d["query_start_loc"].copy_(torch.from_numpy(qsl))
    graph.replay()
    torch.cuda.synchronize()
    compare(y, d["scores"].cpu().numpy())
    assert pkv.get_last_error() == 0


@gpu
def test_weigh_flags_what_does_not_fit(pkvlib):
    """Any int32 as a length or a query start: flagged, nothing else touched."""
    pkv.get_last_error()
    x = batch([64, 100, 30], [1, 2, 2], 8, 2, seed=9)
    for lens in ([64, -1, 30], [64, 2 ** 31 - 1, 30], [64, 1, 30], [64, 16 * x["tables"].shape[1] + 1, 30]):
        d = cuda(x)
        d["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        got = call(x, d)
        assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
        want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE)
        second = np.zeros(x["scores"].shape[0], bool)
        second[x["tables"][1, :7]] = True
        touched = (bound > 0) & ~second[:, None, None]
        assert (np.abs(got - want)[touched] <= bound[touched]).all()
        assert np.array_equal(got[second].view(np.uint32), x["scores"][second].view(np.uint32))
    for qsl in ([0, 1, 2 ** 31 - 1, 5], [0, 1, -2 ** 31, 5], [0, 3, 1, 5], [1, 1, 3, 5]):
        d = cuda(x)
        d["query_start_loc"].copy_(torch.tensor(qsl, dtype=torch.int32))
        call(x, d)
        assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 60])
def test_weigh_bad_pages_are_flagged(pkvlib, rows, fp8):
    """A page id outside the pool: flagged, no score of it is written, and the other sequence is right."""
    pkv.get_last_error()
    x = batch([200, 90], [rows, 1], 8, 2, seed=10, fp8=fp8)
    d = cuda(x)
    d["block_tables"][0, 3] = x["k"].shape[0]
    got = call(x, d)
    assert pkv.get_last_error() == pkv.STATUS_BAD_BLOCK
    want, bound = E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], SCALE, k_scale=x["ks"])
    other = x["tables"][1, :6]
    touched = bound[other] > 0
    assert (np.abs(got[other] - want[other])[touched] <= bound[other][touched]).all()
    bad = x["tables"][0, 3]
    assert np.array_equal(got[bad].view(np.uint32), x["scores"][bad].view(np.uint32))


@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_weigh_offsets_beyond_32_bits(pkvlib, rows):
    """Pages at both ends of a pool of more than 2^31 elements."""
    NB, hkv, hq = 140000, 8, 16
    kc = torch.zeros(NB, hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(NB, hkv, 16, device="cuda")
    table = torch.tensor([[0, NB - 1, 1, NB - 2, 70000, 139000]], dtype=torch.int32, device="cuda")
    x = batch([93], [rows], hq, hkv, seed=11, spare=0)
    pages = table[0].long()
    order = torch.from_numpy(x["tables"][0].astype(np.int64)).cuda()
    d = cuda(x)
    kc[pages], scores[pages] = d["k_cache"][order], d["scores"][order]
    pkv.weigh(d["q"], kc, scores, table, d["seq_lens"], d["query_start_loc"], SCALE)
    got = np.array(x["scores"])
    got[x["tables"][0]] = scores[pages].cpu().numpy()
    compare(x, got)


@gpu
def test_weigh_arguments(pkvlib):
    x = batch([40, 20], [1, 1], 8, 2, seed=12)
    ok = dict(cuda(x), scale=SCALE)
    for error, bad in [(TypeError, dict(q=ok["q"].float())), (ValueError, dict(q=ok["q"][:, :, :64].contiguous())),
                       (ValueError, dict(k_cache=ok["k_cache"].cpu())), (TypeError, dict(scores=ok["scores"].half())),
                       (ValueError, dict(scores=ok["scores"][1:])), (ValueError, dict(seq_lens=ok["seq_lens"][:1])),
                       (TypeError, dict(first=ok["seq_lens"].long())), (ValueError, dict(first=ok["seq_lens"][:1])),
                       (ValueError, dict(scored=ok["seq_lens"].repeat(2))), (TypeError, dict(scale="a")),
                       (TypeError, dict(decay=None)), (pkv.PkvError, dict(decay=-1.0)),
                       (pkv.PkvError, dict(scale=float("nan"))), (TypeError, dict(max_query_len="x")),
                       (pkv.PkvError, dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))),
                       (TypeError, dict(workspace=torch.empty(1 << 20, device="cuda")))]:
        with pytest.raises(error):
            pkv.weigh(**{**ok, **bad})
    desc = pkv.make_desc(ok["k_cache"], 8, ok["block_tables"].shape[1])
    size = pkv.workspace_size_weigh(desc, 2, 2, max_query_len=1, num_keys=80)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert pkv.weigh(**ok, workspace=ws, max_query_len=1, num_keys=80) is None
    compare(x, ok["scores"].cpu().numpy())
    short = torch.empty(max(size - 256, 0), dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.weigh(**ok, workspace=short, max_query_len=1, num_keys=80)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [[1, 2], [1, 90]])
def test_weigh_in_a_graph_and_on_two_streams(pkvlib, rows, fp8):
    """Captured, and replayed with other lengths in the same buffers; then two
    calls at once on two streams, with a workspace each."""
    xs = [batch([600, 333], rows, 8, 2, seed=s, fp8=fp8) for s in (13, 14)]
    ds = [cuda(x) for x in xs]
    fn = pkv.weigh_fp8 if fp8 else pkv.weigh
    fn(scale=SCALE, **cuda(xs[0]))  # first call outside a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(scale=SCALE, **ds[0])
    y = dict(xs[0], lens=np.array([480, 320], np.int32))
    ds[0]["seq_lens"].copy_(torch.tensor([480, 320], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    compare(y, ds[0]["scores"].cpu().numpy())
    ds = [cuda(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for d, stream in zip(ds, streams):
        fn(scale=SCALE, stream=stream, **d)
    torch.cuda.synchronize()
    for x, d in zip(xs, ds):
        compare(x, d["scores"].cpu().numpy())
    assert pkv.get_last_error() == 0
