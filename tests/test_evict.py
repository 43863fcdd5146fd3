"""Eviction by accumulated weight: which rows stay and where they go, exactly,
against the NumPy form."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import eviction as E

gpu = pytest.mark.gpu
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
NULL, ALIGN, SHAPE, RANGE, WORKSPACE = -1, -2, -3, -4, -5


# ---- host -----------------------------------------------------------------------


def test_kept_tokens_by_hand():
    nan, inf = np.nan, np.inf
    s = np.array([5, 1, 3, 3, 9, 0, 3, 2], np.float32)
    assert E.kept_tokens(s, 8, 8, 0, 0).tolist() == list(range(8))
    assert E.kept_tokens(s, 8, 3, 0, 0).tolist() == [0, 2, 4]        # ties: the lowest token
    assert E.kept_tokens(s, 8, 4, 2, 1).tolist() == [0, 1, 4, 7]
    assert E.kept_tokens(s, 8, 3, 5, 5).tolist() == [0, 1, 2]        # the first tokens alone fill the budget
    assert E.kept_tokens(s, 8, 3, 1, 9).tolist() == [0, 6, 7]        # then the recent ones
    assert E.kept_tokens(s, 8, 0, 4, 4).tolist() == []
    assert E.kept_tokens(np.array([nan, -inf, -1, -0.0, 0.0, inf]), 6, 3, 0, 0).tolist() == [3, 4, 5]
    assert E.kept_tokens(np.array([nan, -inf, nan, 1]), 4, 2, 0, 0).tolist() == [0, 3]


def _evict(lib, fp8=False, desc=None, B=4, recent=0, bytes_=1 << 20, **ptr):
    p = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, scores=FAKE, bt=FAKE, sl=FAKE, keep=FAKE, first=FAKE,
             new=FAKE + 4096, ws=FAKE)
    p.update(ptr)
    d = desc or pkv.Desc(64, 16, 2, 8, 128, 16)
    pools = [p["kc"], p["vc"]] + ([p["ks"], p["vs"]] if fp8 else [])
    fn = lib.pkv_evict_fp8 if fp8 else lib.pkv_evict
    return fn(*pools, p["scores"], p["bt"], p["sl"], p["keep"], p["first"], recent, B, p["new"], p["ws"], bytes_,
              ctypes.byref(d), None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), RANGE), (dict(B=2049), RANGE), (dict(recent=-1), RANGE), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(scores=None), NULL), (dict(bt=None), NULL), (dict(sl=None), NULL), (dict(keep=None), NULL),
    (dict(new=None), NULL), (dict(ws=None), NULL), (dict(kc=FAKE + 8), ALIGN), (dict(scores=FAKE + 4), ALIGN),
    (dict(ws=FAKE + 128), ALIGN), (dict(new=FAKE + 4098), ALIGN),
    (dict(new=FAKE), RANGE), (dict(sl=FAKE + 4096 + 12), RANGE), (dict(keep=FAKE + 4096 - 12), RANGE),
    (dict(first=FAKE + 4096), RANGE),
    (dict(desc=pkv.Desc(64, 16, 2, 8, 64, 16)), SHAPE), (dict(desc=pkv.Desc(64, 16, 3, 8, 128, 16)), SHAPE),
    (dict(desc=pkv.Desc(64, 16, 2, 8, 128, 1 << 27)), RANGE), (dict(desc=pkv.Desc(0, 16, 2, 8, 128, 16)), RANGE),
])
def test_evict_refuses(pkvlib, fp8, bad, code):
    before = pkvlib.pkv_launch_count()
    assert _evict(pkvlib, fp8=fp8, **bad) == code
    assert _evict(pkvlib, fp8=fp8, B=0) == 0
    assert pkvlib.pkv_launch_count() == before


def test_evict_workspace_size(pkvlib):
    n = ctypes.c_size_t(0)
    d = pkv.Desc(64, 16, 2, 8, 128, 16)
    size = lambda B: (pkvlib.pkv_evict_workspace_size(ctypes.byref(d), B, ctypes.byref(n)), n.value)
    assert size(3) == (0, 3 * 2 * 16 * 16 * 4) and size(0) == (0, 0)
    assert size(-1)[0] == RANGE and size(2049)[0] == RANGE
    assert pkvlib.pkv_evict_workspace_size(ctypes.byref(d), 3, None) == NULL
    assert pkvlib.pkv_evict_workspace_size(None, 3, ctypes.byref(n)) == NULL


# ---- GPU ------------------------------------------------------------------------


def batch(lens, hkv, seed, fp8=False, width=None, spare=3, kind="weights"):
    """Pools and scores on the host: pages shuffled, unused table entries out of range."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    need = -(-lens // 16)
    NB = int(need.sum()) + spare
    M = width or max(1, int(need.max()))
    tables = np.full((len(lens), M), NB, np.int32)
    perm, at = rng.permutation(NB), 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    shape = (NB, hkv, 16)
    kind_ = np.uint8 if fp8 else np.uint16
    top = 256 if fp8 else 65536
    pools = [rng.integers(0, top, size=shape + (128,), dtype=kind_) for _ in range(2)]
    if fp8:
        pools += [rng.integers(0, 256, size=shape, dtype=np.uint8) for _ in range(2)]
    scores = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        scores = rng.integers(0, 3, size=shape).astype(np.float32)
    if kind == "any":  # every bit pattern: infinities, NaN, negative, subnormal, both zeros
        scores = rng.integers(0, 1 << 32, size=shape, dtype=np.uint32).view(np.float32)
        scores[rng.random(shape) < 0.1] = 0.0
        scores[rng.random(shape) < 0.1] = -0.0
    if kind == "equal":
        scores[:] = 0.25
    return dict(lens=lens, tables=tables, pools=pools, scores=scores, fp8=fp8)


def run(x, keep, first=None, recent=0, **kw):
    """The call's arrays after it, on the host: [pools], scores, new lengths."""
    dev = []
    for p in x["pools"]:
        t = torch.from_numpy(p.view(np.int16) if p.dtype == np.uint16 else p).cuda()
        dev.append(t.view(torch.bfloat16) if p.dtype == np.uint16 else t)
    i32 = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).cuda()
    scores = torch.from_numpy(x["scores"]).cuda()
    args = (*dev, scores, i32(x["tables"]), i32(x["lens"]), i32(keep))
    new = (pkv.evict_fp8 if x["fp8"] else pkv.evict)(*args, first=i32(first), recent=recent, **kw)
    host = [(t if t.dtype == torch.uint8 else t.view(torch.int16)).cpu().numpy() for t in dev]
    return [h.view(p.dtype) for h, p in zip(host, x["pools"])], scores.cpu().numpy(), new.cpu().numpy()


def check(x, keep, first=None, recent=0, flags=0, **kw):
    pools, scores, lens = run(x, keep, first, recent, **kw)
    pe, se, le = E.evict(x["pools"], x["scores"], x["tables"], x["lens"], keep, first, recent)
    assert np.array_equal(lens, le)
    assert np.array_equal(scores.view(np.uint32), se.view(np.uint32))
    for got, want in zip(pools, pe):
        assert np.array_equal(got, want)
    assert pkv.get_last_error() == flags


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["weights", "ties", "any", "equal"])
@pytest.mark.parametrize("lens,keep,first,recent", [
    ([1], [0], None, 0), ([1, 2, 0, 17], [1, 1, 5, 16], None, 0), ([40, 33, 16], [16, 32, 15], [4, 0, 16], 3),
    ([257, 512, 31, 300], [256, 1, 31, 77], [0, 5, 100, 77], 16), ([700, 90], [650, 3], [9, 2], 1000),
    ([1500] * 3, [1499, 700, 64], [0, 699, 8], 7),
])
def test_evict_small(pkvlib, lens, keep, first, recent, kind, fp8):
    x = batch(lens, 2, seed=sum(lens) + recent, fp8=fp8, kind=kind)
    check(x, keep, first, recent)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,hkv,hi,width", [(1, 1, 20000, None), (1, 8, 9000, None), (3, 2, 5000, 1024),
                                               (40, 8, 700, None), (200, 2, 400, 300)])
def test_evict_many_shapes(pkvlib, seqs, hkv, hi, width, fp8):
    """One long sequence (a cluster an item) to many short ones (a CTA an item),
    tables wider than the sequences."""
    rng = np.random.default_rng(seqs + hi)
    lens = rng.integers(0, hi, size=seqs) + (hi // 2 if seqs == 1 else 0)
    keep = rng.integers(0, hi, size=seqs)
    x = batch(lens, hkv, seed=seqs, fp8=fp8, width=width, kind="ties" if seqs == 3 else "weights")
    check(x, keep, rng.integers(0, hi // 4, size=seqs), int(rng.integers(0, hi // 4)))


@gpu
def test_evict_longer_than_a_slice_in_shared_memory(pkvlib):
    """A slice's keys beyond those that shared memory holds are read again."""
    x = batch([150001, 70000], 1, seed=3, kind="ties")
    check(x, [50000, 69999], [1, 0], 100)


@gpu
def test_evict_a_batch_of_long_sequences_on_single_ctas(pkvlib):
    """Items fill the GPU: each of 40,000 tokens is one CTA's."""
    x = batch([40000] + [20] * 159, 2, seed=4, kind="ties")
    check(x, [20001] + [16] * 159, [3] * 160, 5)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hkv", [([4096, 4095, 2500, 300] + [40] * 36, 4), ([4096, 4095, 2500, 300], 2),
                                      ([500, 512, 400, 33], 2), ([9000, 4097], 1)])
@pytest.mark.parametrize("bits", [0, 6, 13, 24])
def test_evict_scores_that_differ_late(pkvlib, lens, hkv, fp8, bits):
    """Scores that agree but for their lowest bits (bits: how many), so that the
    last that stays is told from the next by the third digit, the second or at
    once, with all or a part of what shares a digit staying; on one kernel and two,
    and at the longest tables of one."""
    rng = np.random.default_rng(bits)
    x = batch(lens, hkv, seed=bits + hkv, fp8=fp8)
    low = rng.integers(0, 1 << bits, size=x["scores"].shape, dtype=np.uint32)
    x["scores"] = (np.uint32(0x3E000000) + low).view(np.float32)
    keep = [n // 3 for n in lens]
    check(x, keep, [5] * len(lens), 11)
    half = x["scores"].copy()  # exactly as many larger ones as stay, in the second half
    for b, n in enumerate(lens):
        j = np.arange(n - 11 - (n // 3 - 16), n - 11) if n // 3 > 16 else np.arange(0)
        half[x["tables"][b, j // 16], :, j % 16] += np.float32(1.0)
    check(dict(x, scores=half), keep, [5] * len(lens), 11)


@gpu
@pytest.mark.parametrize("hi", [40, 150])
def test_evict_most_sequences(pkvlib, hi):
    """As many sequences as a call takes."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(0, hi, size=2048)
    x = batch(lens, 1, seed=hi, kind="ties")
    check(x, rng.integers(0, hi, size=2048), rng.integers(0, 9, size=2048), 4)


@gpu
def test_evict_keeps_a_shared_prefix_where_it_is(pkvlib):
    """Two sequences share their first two pages, 32 first tokens."""
    x = batch([100, 132], 2, seed=5)
    x["tables"][1, :2] = x["tables"][0, :2]
    check(x, [50, 40], [32, 32], 4)


@gpu
def test_evict_flags_and_leaves_what_does_not_fit(pkvlib):
    pkv.get_last_error()
    x = batch([100, 90, 80, 70, 60], 2, seed=6)
    good = dict(x)
    x = dict(x, lens=np.array([100, -3, 16 * x["tables"].shape[1] + 1, 70, 2 ** 31 - 1], np.int32))
    keep = np.array([40, 10, 10, -1, 10], np.int32)
    pools, scores, lens = run(x, keep)
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
    assert np.array_equal(lens, [40] + x["lens"][1:].tolist())
    pe, se, _ = E.evict(good["pools"], good["scores"], good["tables"], good["lens"], [40, 90, 80, 70, 60])
    assert np.array_equal(scores, se) and all(np.array_equal(a, b) for a, b in zip(pools, pe))
    pools, scores, lens = run(good, [99, 90, 80, 70, 60], first=[-1, 0, 0, 0, 0])
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY and np.array_equal(lens, good["lens"])
    assert np.array_equal(scores, good["scores"])


@gpu
def test_evict_bad_pages_are_not_touched(pkvlib):
    """Tokens of a page id outside the pool are the first to go, and nothing
    moves onto one; the other heads' and sequences' rows are as they should be."""
    pkv.get_last_error()
    x = batch([96, 50], 2, seed=7)
    tables = x["tables"].copy()
    tables[0, 4] = -2
    y = dict(x, tables=tables)
    pools, scores, lens = run(y, [60, 20])
    assert pkv.get_last_error() == pkv.STATUS_BAD_BLOCK and lens.tolist() == [60, 20]
    low = x["scores"].copy()
    low[x["tables"][0, 4]] = -np.inf
    pe, se, _ = E.evict(x["pools"], low, x["tables"], x["lens"], [60, 20])
    # (of 96 tokens 80 have pages: none of the 60 kept is in the bad one, and none goes there)
    se[x["tables"][0, 4]] = x["scores"][x["tables"][0, 4]]
    assert np.array_equal(scores, se) and all(np.array_equal(a, b) for a, b in zip(pools, pe))


@gpu
def test_evict_offsets_beyond_32_bits(pkvlib):
    """A pool of more than 2^31 elements (and bytes of K alone past 2^32): the
    sequence's pages lie at both of its ends."""
    NB, hkv = 140000, 8
    kc = torch.zeros(NB, hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    scores = torch.zeros(NB, hkv, 16, device="cuda")
    table = torch.tensor([[0, NB - 1, 1, NB - 2, 70000, 139000]], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    pages = table[0].long()
    kc[pages] = torch.randn(6, hkv, 16, 128, generator=gen, device="cuda").to(torch.bfloat16)
    vc[pages] = torch.randn(6, hkv, 16, 128, generator=gen, device="cuda").to(torch.bfloat16)
    scores[pages] = torch.rand(6, hkv, 16, generator=gen, device="cuda")
    host = [t[pages].view(torch.int16).cpu().numpy() for t in (kc, vc)] + [scores[pages].cpu().numpy()]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    new = pkv.evict(kc, vc, scores, table, i32(93), i32(40), recent=3)
    (ke, ve), se, le = E.evict(host[:2], host[2], np.arange(6)[None], np.array([93]), [40], None, 3)
    assert new.tolist() == le.tolist()
    for got, want in zip((kc, vc), (ke, ve)):
        assert np.array_equal(got[pages].view(torch.int16).cpu().numpy(), want)
    assert np.array_equal(scores[pages].cpu().numpy(), se) and pkv.get_last_error() == 0


@gpu
def test_evict_arguments(pkvlib):
    x = batch([40, 20], 2, seed=8)
    as_bf16 = lambda p: torch.from_numpy(p.view(np.int16)).cuda().view(torch.bfloat16)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    ok = dict(k_cache=as_bf16(x["pools"][0]), v_cache=as_bf16(x["pools"][1]), scores=torch.from_numpy(x["scores"]).cuda(),
              block_tables=i32(x["tables"]), seq_lens=i32(x["lens"]), keep=i32([30, 30]))
    for error, bad in [(TypeError, dict(k_cache=ok["k_cache"].float())), (ValueError, dict(v_cache=ok["v_cache"][1:])),
                       (TypeError, dict(scores=ok["scores"].double())), (ValueError, dict(scores=ok["scores"][1:])),
                       (ValueError, dict(scores=ok["scores"].cpu())), (TypeError, dict(keep=ok["keep"].long())),
                       (ValueError, dict(keep=ok["keep"][:1])), (TypeError, dict(keep=None)),
                       (ValueError, dict(first=ok["keep"][:1])), (ValueError, dict(recent=-1)),
                       (TypeError, dict(recent=1.5)), (ValueError, dict(block_tables=ok["block_tables"][:1])),
                       (ValueError, dict(new_lens=ok["keep"][:1].clone())), (pkv.PkvError, dict(new_lens=ok["seq_lens"])),
                       (pkv.PkvError, dict(new_lens=ok["keep"])),
                       (pkv.PkvError, dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
                       (TypeError, dict(workspace=torch.empty(1 << 16, device="cuda")))]:
        with pytest.raises(error):
            pkv.evict(**{**ok, **bad})
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    desc = pkv.make_desc(ok["k_cache"], 2, ok["block_tables"].shape[1])
    ws = torch.empty(pkv.workspace_size_evict(desc, 2), dtype=torch.uint8, device="cuda")
    assert pkv.evict(**ok, new_lens=out, workspace=ws) is out and out.tolist() == [30, 20]
    empty = {**ok, "block_tables": ok["block_tables"][:0], "seq_lens": ok["seq_lens"][:0], "keep": ok["keep"][:0]}
    assert pkv.evict(**empty).numel() == 0


@gpu
def test_evict_in_a_graph_and_on_two_streams(pkvlib):
    """Captured, and replayed on other lengths in the same buffers; then two
    calls at once on two streams, with a workspace each."""
    xs = [batch([600, 333], 2, seed=s, kind="ties") for s in (9, 10)]
    as_bf16 = lambda p: torch.from_numpy(p.view(np.int16)).cuda().view(torch.bfloat16)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    keep, lens2 = i32([100, 300]), np.array([480, 320], np.int32)
    state = [[as_bf16(p) for p in x["pools"]] + [torch.from_numpy(x["scores"]).cuda(), i32(x["tables"]), i32(x["lens"])]
             for x in xs]
    new = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in xs]
    pkv.evict(*[t.clone() for t in state[0]], keep, recent=5)  # first call outside a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.evict(*state[0], keep, recent=5, new_lens=new[0])
    state[0][4].copy_(i32(lens2))
    graph.replay()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    pe, se, le = E.evict(xs[0]["pools"], xs[0]["scores"], xs[0]["tables"], lens2, [100, 300], None, 5)
    assert new[0].tolist() == le.tolist() and np.array_equal(state[0][2].cpu().numpy(), se)
    assert np.array_equal(state[0][0].view(torch.int16).cpu().numpy().view(np.uint16), pe[0])
    state[0] = [as_bf16(p) for p in xs[0]["pools"]] + [torch.from_numpy(xs[0]["scores"]).cuda(), i32(xs[0]["tables"]),
                                                       i32(xs[0]["lens"])]
    torch.cuda.synchronize()
    for st, out, stream in zip(state, new, streams):
        pkv.evict(*st, keep, recent=5, new_lens=out, stream=stream)
    torch.cuda.synchronize()
    for x, st, out in zip(xs, state, new):
        pe, se, le = E.evict(x["pools"], x["scores"], x["tables"], x["lens"], [100, 300], None, 5)
        assert out.tolist() == le.tolist() and np.array_equal(st[2].cpu().numpy(), se)
        for got, want in zip(st, pe):
            assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want)
