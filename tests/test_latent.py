"""attend_latent against float64, element by element within the bound that
oracle.rotary_latent.attend_latent derives."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits
from oracle import rotary_latent as R
from oracle.pkv_oracle import bf16_to_f64

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)


def cuda(a, dtype=None):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a if dtype is None else a.astype(dtype)).cuda()


class Case:
    """A batch over a shuffled pool.  Whatever no query may see is NaN: rows
    past each sequence's end and whole unused pages; unused table entries
    name no page.  Tables ``width`` pages wide or more."""

    def __init__(self, lens, q_lens, H, seed=0, extra_tokens=0, spread=1.0, width=1):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        lens, q_lens = np.asarray(lens), np.asarray(q_lens)
        need = -(-lens // 16)
        nb = int(need.sum()) + 3
        perm = rng.permutation(nb)
        self.tables = np.full((len(lens), max(width, int(need.max()))), nb, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.lens, self.H = lens.astype(np.int32), H
        self.qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        T = int(self.qsl[-1]) + extra_tokens
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.q = (normal(T, H, 576) * spread).to(torch.bfloat16)
        self.pool = torch.full((nb, 16, 576), float("nan"), device="cuda", dtype=torch.bfloat16)
        for b, L in enumerate(lens):
            for i in range(int(need[b])):
                n = min(16, int(L) - 16 * i)
                self.pool[self.tables[b, i], :n] = normal(n, 576).to(torch.bfloat16)

    def args(self):
        return self.q, self.pool, cuda(self.tables), cuda(self.lens), cuda(self.qsl), SCALE

    def expect(self):
        return R.attend_latent(bits(self.q), bits(self.pool), self.tables, self.lens, self.qsl, SCALE)

    def check(self, out, want=None, rows=None):
        o, bound = self.expect() if want is None else want
        got = bf16_to_f64(bits(out))
        n = int(self.qsl[-1])
        err = np.abs(got - o)[:n] - bound[:n]
        assert np.isfinite(got[:n]).all(), f"rows not finite: {np.argwhere(~np.isfinite(got[:n]).all(-1))[:8]}"
        assert (err <= 0).all(), f"{(err > 0).sum()} values beyond the bound, worst by {err.max():.3e}"


CASES = {
    "one_token": ([1], [1], 1),
    "page_edges": ([15, 16, 17, 1], [1, 1, 1, 1], 16),
    "tile_edges": ([63, 64, 65, 128, 129], [1, 1, 1, 1, 1], 12),
    "heads_3": ([100, 7], [1, 1], 3),
    "heads_48": ([300, 65], [1, 1], 48),
    "heads_64": ([300, 65, 640], [1, 1, 1], 64),
    "heads_96": ([200, 31], [1, 1], 96),
    "heads_128": ([500, 64, 1], [1, 1, 1], 128),
    "heads_200": ([130], [1], 200),
    "speculative": ([40, 300, 64, 1000], [2, 5, 3, 4], 20),
    "no_rows": ([40, 0, 64, 9], [1, 0, 0, 1], 16),
    "prompt_alone": ([70], [70], 16),
    "chunk_over_context": ([333, 20], [77, 1], 20),
    "chunk_heads_1": ([200], [200], 1),
    "chunk_heads_128": ([150], [9], 128),
    "split_long": ([9000], [1], 16),
    "split_many": ([5000, 30, 3000, 4097], [1, 1, 2, 1], 64),
}


# Wide tables put sequences of more than 64 rows on pairs of CTAs.
WIDE = 128


@pytest.mark.parametrize("width", [1, WIDE])
@pytest.mark.parametrize("name", CASES)
def test_attend_latent(pkvlib, name, width):
    lens, q_lens, H = CASES[name]
    c = Case(lens, q_lens, H, seed=len(name), width=width)
    out = torch.full((c.q.shape[0], H, 512), float("nan"), device="cuda", dtype=torch.bfloat16)
    got = pkv.attend_latent(*c.args(), out=out, max_query_len=max(q_lens))
    assert got is out
    want = c.expect()
    c.check(out, want)
    assert pkv.get_last_error() == 0
    again = pkv.attend_latent(*c.args(), max_query_len=max(q_lens))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    c.check(pkv.attend_latent(*c.args()), want)  # other tiles where no bound is given


@pytest.mark.parametrize("H,width", [(20, 1), (96, WIDE), (128, WIDE)])
def test_rising_scores_move_the_reference(pkvlib, H, width):
    """Keys that score higher and higher along the sequence: every tile raises
    the reference and rescales what was summed before (one CTA), or the share
    is done again with the maxima known (pairs)."""
    c = Case([1000, 130, 40], [1, 3, 1], H, seed=3, width=width)
    u = torch.randn(576, device="cuda")
    u /= u.norm()
    c.q[:] = (u * 30).to(torch.bfloat16)
    for b, L in enumerate(c.lens):
        for j in range(int(L)):
            c.pool[c.tables[b, j // 16], j % 16] += (u * 0.25 * j).to(torch.bfloat16)
    c.check(pkv.attend_latent(*c.args()))


@pytest.mark.parametrize("H,width", [(16, 1), (128, WIDE)])
def test_falling_and_far_negative_scores(pkvlib, H, width):
    """The first key dominates by far; the rest underflow."""
    c = Case([700], [1], H, seed=4, width=width)
    u = torch.randn(576, device="cuda")
    u /= u.norm()
    c.q[:] = (u * 60).to(torch.bfloat16)
    for j in range(700):
        c.pool[c.tables[0, j // 16], j % 16] -= (u * 0.5 * j + 50).to(torch.bfloat16)
    c.check(pkv.attend_latent(*c.args()))


@pytest.mark.parametrize("H,width", [(12, 1), (72, WIDE)])
def test_rows_behind_the_last_sequence_are_left(pkvlib, H, width):
    c = Case([100, 40], [1, 2], H, seed=5, extra_tokens=5, width=width)
    out = torch.full((8, H, 512), 7.0, device="cuda", dtype=torch.bfloat16)
    pkv.attend_latent(*c.args(), out=out)
    assert bool((out[3:] == 7.0).all())
    c.check(out)


@pytest.mark.parametrize("H,width", [(8, 1), (24, WIDE)])
def test_nan_query_stays_in_its_row(pkvlib, H, width):
    c = Case([300], [4], H, seed=6, width=width)
    c.q[1, 3, 5] = float("nan")
    out = pkv.attend_latent(*c.args())
    assert bool(torch.isnan(out[1, 3]).all())
    c.q[1, 3] = 0
    out[1, 3] = pkv.attend_latent(*c.args())[1, 3]
    c.check(out)


def test_shared_pages_and_long_tables(pkvlib):
    """Two sequences on the same pages, and a table wider than either."""
    c = Case([130, 130], [1, 1], 16, seed=7)
    c.tables = np.concatenate([c.tables, np.full((2, 40), -7, np.int32)], axis=1)
    c.tables[1] = c.tables[0]
    c.check(pkv.attend_latent(*c.args()))


@pytest.mark.parametrize("H,width", [(16, 1), (80, WIDE)])
def test_inconsistent_batches_are_flagged(pkvlib, H, width):
    pkv.get_last_error()
    c = Case([100, 50, 20], [1, 1, 1], H, seed=8, width=width)
    good = c.expect()
    tables = c.tables.copy()
    tables[1, 2] = c.pool.shape[0]  # names no page
    q, pool, _, lens, qsl, scale = c.args()
    out = pkv.attend_latent(q, pool, cuda(tables), lens, qsl, scale)
    assert pkv.get_last_error() == pkv.STATUS_BAD_BLOCK
    got = bf16_to_f64(bits(out))
    assert (np.abs(got - good[0])[[0, 2]] <= good[1][[0, 2]]).all()
    short = c.lens.copy()
    short[1] = 0  # fewer tokens than queries
    out = torch.full((3, H, 512), 7.0, device="cuda", dtype=torch.bfloat16)
    pkv.attend_latent(q, pool, cuda(c.tables), cuda(short), qsl, scale, out=out)
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
    assert bool((out[1] == 7.0).all())
    got = bf16_to_f64(bits(out))
    assert (np.abs(got - good[0])[[0, 2]] <= good[1][[0, 2]]).all()


@pytest.mark.parametrize("B,longest,joined", [(38, 512, False), (38, 513, True), (39, 512, True), (1, 512, False)])
def test_short_batches_are_not_joined(pkvlib, B, longest, joined):
    """Few sequences of at most 512 tokens are cut nowhere, so no kernel joins
    pieces; one sequence or one token more, and it runs."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the bounds are those of 152 SMs")
    c = Case([longest] + [512 - 13 * (b % 39) for b in range(1, B)], [1] * B, 16, seed=B)
    c.check(pkv.attend_latent(*c.args(), max_query_len=1))
    with pkv.Trace(8) as tr:
        pkv.attend_latent(*c.args(), max_query_len=1)
    torch.cuda.synchronize()
    assert tr.read("latent")[1] == 1 and tr.read("merge")[1] == int(joined)
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("H,width", [(16, 1), (96, WIDE)])
def test_any_int32_as_length_or_query_start(pkvlib, H, width):
    """Lengths and query starts whose sums or differences leave int32 are
    inconsistent like any other: the sequence is skipped, its neighbours are
    not."""
    pkv.get_last_error()
    c = Case([100, 50, 20], [1, 1, 1], H, seed=12, width=width)
    good = c.expect()
    q, pool, tables, lens, qsl, scale = c.args()
    top = 2**31 - 1
    for at, value in ((1, top), (1, top - 7), (1, -2**31), (1, tables.shape[1] * 16 + 1)):
        L = c.lens.copy()
        L[at] = value
        out = torch.full((3, H, 512), 7.0, device="cuda", dtype=torch.bfloat16)
        pkv.attend_latent(q, pool, tables, cuda(L), qsl, scale, out=out)
        assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
        assert bool((out[1] == 7.0).all())
        got = bf16_to_f64(bits(out))
        assert (np.abs(got - good[0])[[0, 2]] <= good[1][[0, 2]]).all()
    for value in (top, -2**31):  # the end of the second sequence and the start of the third
        starts = c.qsl.copy()
        starts[2] = value
        out = torch.full((3, H, 512), 7.0, device="cuda", dtype=torch.bfloat16)
        pkv.attend_latent(q, pool, tables, lens, cuda(starts), scale, out=out)
        assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
        assert bool((out[1:] == 7.0).all())
        got = bf16_to_f64(bits(out))
        assert (np.abs(got - good[0])[0] <= good[1][0]).all()


def test_two_graphs_share_a_workspace_and_a_stream_of_its_own(pkvlib):
    cases = [Case([3000, 200], [1, 1], 16, seed=9), Case([70, 2500, 5], [3, 1, 1], 64, seed=10),
             Case([900, 2100], [1, 1], 128, seed=11)]
    size = max(pkv.workspace_size_latent(pkv.make_latent_desc(c.pool, c.H, c.tables.shape[1]), len(c.lens), c.q.shape[0])
               for c in cases)
    ws = torch.full((size,), 255, device="cuda", dtype=torch.uint8)
    args, outs, graphs = [c.args() for c in cases], [], []
    for c, a in zip(cases, args):
        out = torch.zeros(c.q.shape[0], c.H, 512, device="cuda", dtype=torch.bfloat16)
        pkv.attend_latent(*a, out=out, workspace=ws)  # first call outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.attend_latent(*a, out=out, workspace=ws)
        outs.append(out)
        graphs.append(g)
    wants = [c.expect() for c in cases]
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        for c, o, w in zip(cases, outs, wants):
            c.check(o, w)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [pkv.attend_latent(*a, stream=stream) for a in args]
    stream.synchronize()
    for c, o, w in zip(cases, got, wants):
        c.check(o, w)


@pytest.mark.parametrize("lens,H,width", [([3000, 200, 77], 16, 1), ([3000, 900, 77], 96, WIDE), ([70, 200, 77], 16, 1)])
def test_a_workspace_shared_with_the_other_attention(pkvlib, lens, H, width):
    """One scratch buffer behind both attention calls of a stream: each may
    begin before the other has ended, and neither touches it before that."""
    pkv.get_last_error()
    c = Case(lens, [1, 1, 1], H, seed=15, width=width)
    args = c.args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(15)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    q, kc, vc = normal(3, 32, 128), normal(c.pool.shape[0], 8, 16, 128), normal(c.pool.shape[0], 8, 16, 128)
    other = (q, kc, vc, *args[2:5], 0.088)
    want, want_other = pkv.attend_latent(*args), pkv.attend(*other, max_query_len=1)
    c.check(want)
    size = max(pkv.workspace_size_latent(pkv.make_latent_desc(c.pool, H, c.tables.shape[1]), 3, 3),
               pkv.workspace_size(pkv.make_desc(kc, 32, c.tables.shape[1]), 3, 3))
    ws = torch.full((size,), 255, device="cuda", dtype=torch.uint8)
    got = []
    for _ in range(20):
        got.append((pkv.attend_latent(*args, workspace=ws), pkv.attend(*other, workspace=ws, max_query_len=1)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a.view(torch.int16), want.view(torch.int16))
        torch.testing.assert_close(b.float(), want_other.float(), rtol=2**-7, atol=1e-2)
    assert pkv.get_last_error() == 0


def test_lengths_written_right_before_each_call(pkvlib):
    """A decode loop whose lengths, tables and queries are device results of
    the operations right before the call, eager and captured."""
    pkv.get_last_error()
    for H, width in ((16, 1), (96, WIDE)):
        c = Case([700, 400, 90], [1, 1, 1], H, seed=16, width=width)
        q, pool, tables, _, qsl, scale = c.args()
        lens = torch.zeros(3, dtype=torch.int32, device="cuda")
        steps = [cuda(np.array(x, np.int32)) for x in ([700, 1, 33], [5, 400, 90], [699, 17, 64], [1, 1, 1])]
        moved = torch.empty_like(tables)
        want = [pkv.attend_latent(q, pool, tables, x, qsl, scale) for x in steps]
        torch.cuda.synchronize()

        def loop(outs):
            for x, out in zip(steps, outs):
                lens.copy_(x * 2 - x)
                moved.copy_(tables)
                pkv.attend_latent(q * 1, pool, moved, lens + 0, qsl, scale, out=out)
                moved.fill_(-1)  # behind the call: it has read them

        outs = [torch.empty_like(w) for w in want]
        for _ in range(5):
            loop(outs)
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), w.view(torch.int16)) for o, w in zip(outs, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loop(outs)
        for _ in range(5):
            for o in outs:
                o.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), w.view(torch.int16)) for o, w in zip(outs, want))
    assert pkv.get_last_error() == 0


def test_calls_at_once_on_two_streams(pkvlib):
    """Both kernels fill an SM each; calls on two streams share the GPU and
    nothing else."""
    pkv.get_last_error()
    cases = [Case([3000, 200, 77], [1, 1, 1], 16, seed=13), Case([900, 2100], [2, 1], 96, seed=14, width=WIDE)]
    args = [c.args() for c in cases]
    want = [pkv.attend_latent(*a) for a in args]
    for c, w in zip(cases, want):
        c.check(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(12):
        for k in (i & 1, 1 - (i & 1)):
            got[k].append(pkv.attend_latent(*args[k], stream=streams[k]))  # a workspace of its own each call
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            assert torch.equal(g.view(torch.int16), want[k].view(torch.int16))
    assert pkv.get_last_error() == 0


def test_a_step_appends_and_attends(pkvlib):
    """Three steps as a model with latent attention makes them, the last one
    speculative: write_latent, then attend_latent right behind it."""
    from test_rope import table
    H, B, P = 20, 3, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    tab = table(512, 64)
    tables = np.random.default_rng(1).permutation(30).reshape(B, 10).astype(np.int32)
    pool = torch.full((30, P, 576), float("nan"), device="cuda", dtype=torch.bfloat16)
    ref = bits(pool)
    lens = np.zeros(B, np.int64)
    for q_lens in ([40, 1, 130], [1, 1, 1], [2, 4, 3]):
        qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        T = int(qsl[-1])
        pos = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, q_lens)])
        seq = np.repeat(np.arange(B), q_lens)
        slots = tables[seq, pos // P].astype(np.int64) * P + pos % P
        lens = lens + q_lens
        kv_a, qp, q = normal(T, 576), normal(T, H, 192), normal(T, H, 576)
        meta = cuda(tables), cuda(lens, np.int32), cuda(qsl)
        want_q = bits(q)
        pkv.write_latent(kv_a[:, :512], kv_a[:, 512:], cuda(pos), cuda(tab), cuda(slots), pool, q_pe=qp[..., 128:],
                         q_out=q, interleaved=True)
        out = pkv.attend_latent(q, pool, *meta, SCALE, max_query_len=max(q_lens))
        ref = R.write_latent(bits(kv_a[:, :512]), bits(kv_a[:, 512:]), pos, tab, slots, ref, True)
        want_q[..., 512:] = R.rotate_bits(bits(qp[..., 128:]), pos, tab, True)
        o, bound = R.attend_latent(want_q, ref, tables, lens, qsl, SCALE)
        err = np.abs(bf16_to_f64(bits(out)) - o)
        assert np.array_equal(bits(q), want_q) and (err <= bound).all()
    assert pkv.get_last_error() == 0


def test_rotated_append_then_attend(pkvlib):
    """write_rope feeding attend, against the oracle's attention over rotated
    rows: decode rows and a prompt chunk, queries rotated by the same call."""
    from helpers import MAX_ABS_TOL, MEAN_ABS_TOL, to_device
    from oracle.pkv_oracle import attend, write
    from test_rope import table
    from workloads import make_batch
    b = make_batch([17, 64, 100, 255, 300], [1, 1, 1, 1, 40], 32, 8, seed=12, device="cuda")
    meta = to_device(b)
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(b.seq_lens, b.q_lens)]).astype(np.int64)
    tab = table(512, 128)
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    q = pkv.write_rope(b.k_new, b.v_new, cuda(pos), cuda(tab), meta["slot_mapping"], kc, vc, q=b.q)
    out = pkv.attend(q, kc, vc, meta["block_tables"], meta["seq_lens"], meta["query_start_loc"], b.scale)
    k_ref, v_ref = write(R.rotate_bits(bits(b.k_new), pos, tab, False), bits(b.v_new), b.slot_mapping,
                         bits(b.k_cache), bits(b.v_cache), 16)
    ref = attend(R.rotate_bits(bits(b.q), pos, tab, False), k_ref, v_ref, b.block_tables, b.seq_lens,
                 b.query_start_loc, b.scale, 32, 8, 16)
    err = np.abs(bf16_to_f64(bits(out)) - ref)
    assert err.max() <= MAX_ABS_TOL and err.mean() <= MEAN_ABS_TOL


@pytest.mark.parametrize("H,width", [(5, 1), (64, 1), (128, WIDE)])
def test_the_same_bits_many_times(pkvlib, H, width):
    """Calls right behind each other on one workspace: nothing of a result may
    depend on when a CTA or a copy was ready."""
    c = Case([2300, 17, 640, 1, 64, 1025, 333], [1, 2, 1, 1, 3, 1, 1], H, seed=12, width=width)
    args = c.args()
    ws = torch.zeros(pkv.workspace_size_latent(pkv.make_latent_desc(c.pool, H, c.tables.shape[1]), 7, c.q.shape[0]),
                     dtype=torch.uint8, device="cuda")
    outs = [pkv.attend_latent(*args, workspace=ws, max_query_len=3) for _ in range(200)]
    c.check(outs[0])
    assert all(torch.equal(outs[0].view(torch.int16), o.view(torch.int16)) for o in outs)
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(pkvlib, seed):
    rng = np.random.default_rng(100 + seed)
    B, H = int(rng.integers(1, 12)), int(rng.integers(1, 257))
    lens = np.round(np.exp(rng.uniform(0, np.log(3000), B))).astype(int)
    most = int(rng.choice([1, 1, 4, 60]))
    q_lens = np.minimum(rng.integers(0 if B > 1 else 1, most, size=B, endpoint=True), lens)
    if q_lens.sum() == 0:
        q_lens[0] = 1
    c = Case(lens, q_lens, H, seed=seed, width=int(rng.choice([1, WIDE])))
    bound = int(rng.choice([0, 1, int(q_lens.max()), 1000]))  # a wrong bound changes tiles, not results
    c.check(pkv.attend_latent(*c.args(), max_query_len=bound))
    assert pkv.get_last_error() == 0
