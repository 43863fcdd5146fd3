"""A decode loop as a server captures it: one graph whose lengths, positions,
slots and block tables are updated in place by the step itself, right before
the append and the attention that read them."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from test_latent import SCALE, cuda
from test_rope import table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,pages", [(16, 6), (16, 130), (96, 130)])
def test_a_captured_decode_loop_in_place(pkvlib, H, pages):
    """Sequences start at lengths around a page's and a tile's end and grow by a
    token a replay; a new page is taken from the spare ones when one is full.
    Every step against the same calls made one by one, with the device idle in
    between and on memory of their own."""
    pkv.get_last_error()
    B, steps = 5, 70
    rng = np.random.default_rng(71)
    start = np.array([1, 15, 60, 63, 17])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(71)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    nb = 60
    all_pages = cuda(rng.permutation(nb).reshape(B, nb // B).astype(np.int32))
    tables = torch.full((B, pages), nb, device="cuda", dtype=torch.int32)
    used = min(pages, nb // B)
    pool0 = normal(nb, 16, 576)
    pool, lens = pool0.clone(), cuda(start.astype(np.int32))
    qsl, tab = cuda(np.arange(B + 1, dtype=np.int32)), cuda(table(512, 64))
    seq = torch.arange(B, device="cuda")
    noise = normal(steps, B, 576)
    queries = normal(steps, B, H, 640)
    step = torch.zeros(1, device="cuda", dtype=torch.int64)
    kv, qx = torch.empty(B, 576, device="cuda", dtype=torch.bfloat16), torch.empty(B, H, 640, device="cuda", dtype=torch.bfloat16)
    pos, slots = (torch.empty(B, device="cuda", dtype=torch.int64) for _ in range(2))
    q, out = (torch.empty(B, H, n, device="cuda", dtype=torch.bfloat16) for n in (576, 512))
    ws = torch.empty(pkv.workspace_size_latent(pkv.make_latent_desc(pool, H, pages), B, B), dtype=torch.uint8, device="cuda")

    def one():
        kv.copy_(noise[step][0])
        qx.copy_(queries[step][0])
        q.copy_(qx[..., :576])
        pos.copy_(lens)
        lens.add_(1)
        tables[:, :used] = torch.where((torch.arange(used, device="cuda") * 16 < lens[:, None]), all_pages[:, :used], nb)
        slots.copy_(all_pages[seq, pos // 16].long() * 16 + pos % 16)
        pkv.write_latent(kv[:, :512], kv[:, 512:], pos, tab, slots, pool, q_pe=qx[..., 576:], q_out=q)
        pkv.attend_latent(q, pool, tables, lens, qsl, SCALE, out=out, workspace=ws, max_query_len=1)
        step.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one()
    pool.copy_(pool0)
    lens.copy_(cuda(start.astype(np.int32)))
    tables.fill_(nb)
    step.zero_()
    outs = torch.empty(steps, B, H, 512, device="cuda", dtype=torch.bfloat16)
    grow = min(steps, used * 16 - int(start.max()))
    for i in range(grow):
        g.replay()
        outs[i].copy_(out)
    torch.cuda.synchronize()
    cache = pool0.clone()
    for i in range(grow):
        L = start + i + 1
        t = all_pages[:, :used].clone()
        t = torch.cat([torch.where(torch.arange(used, device="cuda") * 16 < cuda(L)[:, None], t, nb).int(),
                       torch.full((B, pages - used), nb, device="cuda", dtype=torch.int32)], dim=1)
        p = cuda(L - 1)
        s = all_pages[seq, p // 16].long() * 16 + p % 16
        qi = queries[i][..., :576].contiguous()
        torch.cuda.synchronize()
        pkv.write_latent(noise[i][:, :512], noise[i][:, 512:], p, tab, s, cache, q_pe=queries[i][..., 576:], q_out=qi)
        torch.cuda.synchronize()
        want = pkv.attend_latent(qi, cache, t, cuda(L.astype(np.int32)), qsl, SCALE, max_query_len=1)
        torch.cuda.synchronize()
        assert torch.equal(outs[i].view(torch.int16), want.view(torch.int16)), i
    assert torch.equal(pool.view(torch.int16), cache.view(torch.int16))
    assert grow > 30 and pkv.get_last_error() == 0


def test_calls_from_several_threads(pkvlib):
    """A thread a stream, each with its own step of append and attention; the
    calls run without the interpreter's lock."""
    import threading

    from test_latent import WIDE, Case
    pkv.get_last_error()
    cases = [Case([300, 77, 1500], [1, 1, 1], 16, seed=81), Case([300, 900], [2, 1], 96, seed=82, width=WIDE),
             Case([64, 65, 9], [1, 3, 1], 20, seed=83), Case([2100], [1], 64, seed=84)]
    args = [c.args() for c in cases]
    want = [pkv.attend_latent(*a) for a in args]
    for c, w in zip(cases, want):
        c.check(w)
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [pkv.attend_latent(*args[k]) for _ in range(100)]
                stream.synchronize()
            if not all(torch.equal(g.view(torch.int16), want[k].view(torch.int16)) for g in got):
                failed.append(k)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and pkv.get_last_error() == 0
