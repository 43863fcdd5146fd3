"""The operators of an engine that keeps its caches small, one behind the other:
a prompt of image patches is appended with positions on three axes, its last
rows weigh it, it is cut down, and decode steps append, attend and weigh on what
is left and cut it down again, all on the same pages, tables and lengths, without
the host reading anything back."""

import numpy as np
import pytest
import torch

import oracle.pkv_oracle as O
import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits, compare
from oracle import eviction as E
from oracle import rotary_latent as R
from oracle.pkv_oracle import bf16_to_f64
from test_rope import cuda, table
from test_rope_axes import rows_of

gpu = pytest.mark.gpu
HQ, HKV, SCALE = 8, 2, 128 ** -0.5
AXES = [i % 3 for i in range(64)]


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def close(got, want, bound):
    touched = bound > 0
    assert (np.abs(got - want)[touched] <= bound[touched]).all()
    assert np.array_equal(got[~touched].view(np.uint32), want[~touched].astype(np.float32).view(np.uint32))


@gpu
@pytest.mark.parametrize("graphs", [False, True])
def test_append_weigh_evict_attend(pkvlib, graphs):
    """Against the same steps of the NumPy forms.  The oracle's eviction goes by
    the device's scores (a score off by its last bits may change which token
    stays), which are compared with the oracle's first."""
    pkv.get_last_error()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rng = np.random.default_rng(3)
    lens, keep, first, recent, steps = [230, 57, 400], [64, 64, 100], [4, 0, 16], 8, 3
    window = 16
    B, NB = len(lens), 64
    tables = np.full((B, 32), NB, np.int32)
    perm, at = rng.permutation(NB), 0
    for b, L in enumerate(lens):
        need = -(-(L + steps) // 16)
        tables[b, :need] = perm[at:at + need]
        at += need
    tab = table(512, 128)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    kc, vc, scores = normal(gen, NB, HKV, 16, 128), normal(gen, NB, HKV, 16, 128), torch.full((NB, HKV, 16), float("nan"),
                                                                                             device="cuda")
    d_tables, d_first, d_keep, d_tab = i32(tables), i32(first), i32(keep), cuda(tab)
    k_ref, v_ref, s_ref = bits(kc), bits(vc), scores.cpu().numpy()

    # ---- prompts ----
    T = sum(lens)
    qsl = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = normal(gen, T, HQ, 128), normal(gen, T, HKV, 128), normal(gen, T, HKV, 128)
    positions = np.concatenate([np.stack([np.arange(L) // 64, np.arange(L) // 8 % 8, np.arange(L) % 8]) for L in lens], axis=1)
    slots = np.concatenate([tables[b, np.arange(L) // 16] * 16 + np.arange(L) % 16 for b, L in enumerate(lens)])
    turned = pkv.write_rope_axes(k, v, cuda(positions), bytes(AXES), d_tab, cuda(slots.astype(np.int64)), kc, vc, q=q)
    rows = rows_of(tab, positions, AXES)
    turn = lambda b, r: R.f64_to_bf16(R.rotate(bf16_to_f64(b), r, False))
    k_ref, v_ref = O.write(turn(bits(k), rows), bits(v), slots, k_ref, v_ref, 16)
    q_ref = turn(bits(q), rows)
    d_lens = i32(lens)
    out = pkv.attend(turned, kc, vc, d_tables, d_lens, i32(qsl), SCALE)
    compare(out, O.attend(q_ref, k_ref, v_ref, tables, lens, qsl, SCALE, HQ, HKV, 16), what="prompt")
    # the last rows of each prompt judge all of it
    pick = np.concatenate([np.arange(qsl[b + 1] - window, qsl[b + 1]) for b in range(B)])
    starts = np.arange(B + 1) * window
    pkv.weigh(turned[cuda(pick)].contiguous(), kc, scores, d_tables, d_lens, i32(starts), SCALE, decay=0.0,
              first=d_first, max_query_len=window)
    want, bound = E.weigh(q_ref[pick], k_ref, s_ref, tables, lens, starts, SCALE, 0.0, first)
    s_dev = scores.cpu().numpy()
    close(s_dev, want, bound)
    d_lens = pkv.evict(kc, vc, scores, d_tables, d_lens, d_keep, first=d_first, recent=recent)
    (k_ref, v_ref), s_ref, lens = E.evict([k_ref, v_ref], s_dev, tables, lens, keep, first, recent)
    assert d_lens.tolist() == lens.tolist()
    assert np.array_equal(bits(kc), k_ref) and np.array_equal(bits(vc), v_ref)

    # ---- decode steps: text tokens, all axes alike; positions go on counting ----
    text = np.array([230, 57, 400])
    step_q, step_k, step_v = normal(gen, B, HQ, 128), normal(gen, B, HKV, 128), normal(gen, B, HKV, 128)
    d_pos = torch.zeros(B, dtype=torch.int64, device="cuda")
    d_slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    d_starts = i32(np.arange(B + 1))
    next_lens = d_lens.clone()
    seq = torch.arange(B, device="cuda")
    rotated, outs = torch.empty_like(step_q), torch.empty_like(step_q)

    def step():
        # where the next token goes, on the device: lengths differ from those the host knows of
        d_slots.copy_(d_tables[seq, (next_lens // 16).long()].long() * 16 + next_lens % 16)
        pkv.write_rope_axes(step_k, step_v, d_pos.expand(3, -1), bytes(AXES), d_tab, d_slots, kc, vc, q=step_q, q_out=rotated)
        next_lens.add_(1)
        pkv.attend(rotated, kc, vc, d_tables, next_lens, d_starts, SCALE, out=outs, max_query_len=1)
        pkv.weigh(rotated, kc, scores, d_tables, next_lens, d_starts, SCALE, decay=0.5, first=d_first, max_query_len=1)
        d_lens.copy_(next_lens)
        pkv.evict(kc, vc, scores, d_tables, d_lens, d_keep, first=d_first, recent=recent, new_lens=next_lens)

    run = step
    if graphs:
        graph = torch.cuda.CUDAGraph()
        saved = [t.clone() for t in (kc, vc, scores, next_lens, d_lens)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # allocations of a first run
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step()
        for t, old in zip((kc, vc, scores, next_lens, d_lens), saved):
            t.copy_(old)
        run = graph.replay
    for i in range(steps):
        for t in (step_q, step_k, step_v):
            t.copy_(normal(gen, *t.shape))
        d_pos.copy_(torch.from_numpy(text + i))
        run()
        torch.cuda.synchronize()
        rows = rows_of(tab, np.stack([text + i] * 3), AXES)
        slots = tables[np.arange(B), lens // 16] * 16 + lens % 16
        k_ref, v_ref = O.write(turn(bits(step_k), rows), bits(step_v), slots, k_ref, v_ref, 16)
        q_ref = turn(bits(step_q), rows)
        lens = lens + 1
        starts = np.arange(B + 1)
        compare(outs, O.attend(q_ref, k_ref, v_ref, tables, lens, starts, SCALE, HQ, HKV, 16), what=f"step {i}")
        want, bound = E.weigh(q_ref, k_ref, s_ref, tables, lens, starts, SCALE, 0.5, first)
        # the device has evicted already: its scores against the oracle's, kept by the oracle's (ties of
        # nearly equal scores are the oracle's business here: none lies within the bound)
        for b in range(B):
            if lens[b] > keep[b]:
                token = np.arange(lens[b])
                for h in range(HKV):
                    page = tables[b, token // 16]
                    s, e = want[page, h, token % 16], bound[page, h, token % 16]
                    middle = np.arange(first[b], lens[b] - recent)
                    order = middle[np.argsort(-s[middle], kind="stable")]
                    cut = keep[b] - first[b] - recent
                    assert s[order[cut - 1]] - s[order[cut]] > e[order[cut - 1]] + e[order[cut]]
        before = lens
        (k_ref, v_ref, bound), s_ref, lens = E.evict([k_ref, v_ref, bound], want, tables, before, keep, first, recent)
        assert next_lens.tolist() == lens.tolist() and d_lens.tolist() == before.tolist()
        assert np.array_equal(bits(kc), k_ref) and np.array_equal(bits(vc), v_ref)
        s_dev = scores.cpu().numpy()
        live = bound > 0
        assert (np.abs(s_dev - s_ref)[live] <= bound[live]).all()
        s_ref = s_dev  # rounding does not add up over the steps
    assert pkv.get_last_error() == 0
