"""Offsets that pass 32 bits: pools, queries and results of more than 2^31
elements, and sequences of a million tokens and more."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits
from oracle import rotary_latent as R
from test_latent import SCALE, WIDE, Case, cuda
from test_rope import table

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("H,width", [(16, 1), (96, WIDE)])
def test_pages_far_into_the_pool(pkvlib, H, width):
    """Pages spread over a pool of 2.8e9 elements, the last one among them."""
    c = Case([700, 33, 130], [1, 2, 1], H, seed=61, width=width)
    small, nb = c.pool, 300000
    want = c.expect()
    where = np.linspace(0, nb - 1, small.shape[0]).astype(np.int64)
    c.pool = torch.empty(nb, 16, 576, device="cuda", dtype=torch.bfloat16)
    c.pool[cuda(where)] = small
    live = c.tables < small.shape[0]
    c.tables = np.where(live, where[np.where(live, c.tables, 0)], nb).astype(np.int32)
    assert int(c.tables[live].max()) * 16 * 576 > 2**31
    c.check(pkv.attend_latent(*c.args(), max_query_len=2), want)
    assert pkv.get_last_error() == 0


def test_appends_far_into_the_pool(pkvlib):
    nb, T = 300000, 40
    pos, tab = np.arange(T) * 3, table(256, 64)
    slots = np.random.default_rng(1).permutation(nb * 16)[:T]
    slots[-1] = nb * 16 - 1
    c, k = normal(1, T, 512), normal(2, T, 64)
    pool = torch.empty(nb, 16, 576, device="cuda", dtype=torch.bfloat16)
    pkv.write_latent(c, k, cuda(pos), cuda(tab), cuda(slots), pool)
    rows = pool.view(-1, 576)[cuda(slots)]
    assert np.array_equal(bits(rows[:, :512]), bits(c))
    assert np.array_equal(bits(rows[:, 512:]), R.rotate_bits(bits(k[:, None]), pos, tab, False)[:, 0])
    del pool
    nb, hkv, tab = 180000, 8, table(256, 128)
    slots = np.random.default_rng(2).permutation(nb * 16)[:T]
    slots[-1] = nb * 16 - 1
    kv = normal(3, T, 2 * hkv, 128)
    kc, vc = (torch.empty(nb, hkv, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pkv.write_rope(kv[:, :hkv], kv[:, hkv:], cuda(pos), cuda(tab), cuda(slots), kc, vc)
    page, row = cuda(slots // 16), cuda(slots % 16)
    assert np.array_equal(bits(kc[page, :, row]), R.rotate_bits(bits(kv[:, :hkv]), pos, tab, False))
    assert np.array_equal(bits(vc[page, :, row]), bits(kv[:, hkv:]))
    assert pkv.get_last_error() == 0


def test_queries_of_more_than_2_31_elements(pkvlib):
    """q_out and the results of a step whose queries do not fit 32-bit offsets."""
    T, hq, hkv = 530000, 32, 2
    pos, tab = np.arange(T) % 200, table(200, 128)
    x = normal(4, T, hq + 2 * hkv, 128)
    kc, vc = (torch.empty(1, hkv, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = pkv.write_rope(x[:, hq:hq + hkv], x[:, hq + hkv:], cuda(pos), cuda(tab), cuda(np.full(T, -1)), kc, vc, q=x[:, :hq])
    assert q.numel() > 2**31
    at = np.r_[0:50, T // 2:T // 2 + 50, T - 50:T]
    assert np.array_equal(bits(q[cuda(at)]), R.rotate_bits(bits(x[cuda(at), :hq]), pos[at], tab, False))
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("H,width", [(64, 1), (128, WIDE)])
def test_results_of_more_than_2_31_elements(pkvlib, H, width):
    """The rows in use lie at both ends of q and out; the sequence between them
    has more queries than tokens, and is flagged and skipped."""
    T = 2**31 // (512 * H) + 300
    c = Case([50, 64, 200], [50, 0, 40], H, seed=62, width=width)
    want, bound = c.expect()
    q = torch.zeros(T, H, 576, device="cuda", dtype=torch.bfloat16)
    q[:50], q[T - 40:] = c.q[:50], c.q[50:]
    c.qsl = np.array([0, 50, T - 40, T], np.int32)
    out = torch.full((T, H, 512), 7.0, device="cuda", dtype=torch.bfloat16)
    assert out.numel() > 2**31
    pkv.attend_latent(q, *c.args()[1:], out=out)
    assert pkv.get_last_error() == pkv.STATUS_BAD_QUERY
    got = torch.cat([out[:50], out[T - 40:]]).double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all()
    assert bool((out[50:T - 40:997] == 7.0).all())


@pytest.mark.parametrize("H", [16, 128])
def test_a_million_and_a_half_tokens(pkvlib, H):
    """One sequence, cut among all SMs; in float64 with the bound of
    oracle.rotary_latent.attend_latent."""
    L = 1_500_001
    nb = -(-L // 16)
    pool, q = normal(63, nb, 16, 576), normal(64, 1, H, 576)
    table_ = np.random.default_rng(63).permutation(nb).astype(np.int32)[None]
    out = pkv.attend_latent(q, pool, cuda(table_), cuda(np.array([L], np.int32)), cuda(np.array([0, 1], np.int32)), SCALE,
                            max_query_len=1)
    rows = pool[cuda(table_[0]).long()].view(-1, 576)[:L]
    top = torch.full((H,), -float("inf"), device="cuda", dtype=torch.float64)
    terms = torch.zeros(H, device="cuda", dtype=torch.float64)
    for part in rows.split(250000):
        k = part.double()
        top = torch.maximum(top, (SCALE * (q[0].double() @ k.T)).amax(1))
        terms = torch.maximum(terms, (SCALE * (q[0].double().abs() @ k.abs().T)).amax(1))
    total, o, mags = 0, 0, 0
    for part in rows.split(250000):
        k = part.double()
        w = torch.exp(SCALE * (q[0].double() @ k.T) - top[:, None])
        total, o, mags = total + w.sum(1), o + w @ k[:, :512], mags + w @ k[:, :512].abs()
    o, mags = o / total[:, None], mags / total[:, None]
    rel = 2.0 ** -8 + 576 * 2.0 ** -23 * terms + 2.0 ** -20
    bound = (2.0 ** -8 * o.abs() + rel[:, None] * (mags + o.abs())) * (1 + 2.0 ** -6) + 1e-30
    assert bool(((out[0].double() - o).abs() <= bound).all())
    assert pkv.get_last_error() == 0
