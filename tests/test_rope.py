"""Appends that rotate on the way: bit for bit against the NumPy form (the
rotation is defined in fp32 arithmetic and rounded once)."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits
from oracle import rotary_latent as R
from oracle.pkv_oracle import bf16_to_f64, write, write_fp8

gpu = pytest.mark.gpu


def table(max_pos, dim, base=10000.0):
    freq = base ** (-np.arange(0, dim, 2) / dim)
    angle = np.arange(max_pos)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def inputs(T, hq, hkv, rot, seed, max_pos=512, strided=True, pages=None):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    pages = pages or -(-T // 16) + 2
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    qkv = normal(T, hq + 2 * hkv, 128)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    positions = rng.integers(0, max_pos, size=T)
    slots = rng.permutation(pages * 16)[:T]
    return dict(q=q, k=k, v=v, positions=positions, slots=slots, table=table(max_pos, rot),
                kc=normal(pages, hkv, 16, 128), vc=normal(pages, hkv, 16, 128))


def call(x, interleaved, slots=None, **kw):
    kc, vc = x["kc"].clone(), x["vc"].clone()
    q = pkv.write_rope(x["k"], x["v"], cuda(x["positions"]), cuda(x["table"]),
                       cuda(x["slots"] if slots is None else slots), kc, vc, interleaved=interleaved, **kw)
    return q, kc, vc


def expect(x, interleaved, slots=None):
    k = R.rotate_bits(bits(x["k"]), x["positions"], x["table"], interleaved)
    kc, vc = write(k, bits(x["v"]), x["slots"] if slots is None else slots, bits(x["kc"]), bits(x["vc"]), 16)
    return R.rotate_bits(bits(x["q"]), x["positions"], x["table"], interleaved), kc, vc


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,rot", [(1, 32, 8, 128), (1, 1, 1, 16), (3, 8, 8, 64), (17, 16, 1, 96),
                                          (129, 32, 2, 48), (1120, 8, 2, 128), (2500, 4, 4, 32)])
def test_write_rope_bits(pkvlib, T, hq, hkv, rot, interleaved):
    x = inputs(T, hq, hkv, rot, seed=T + rot)
    q, kc, vc = call(x, interleaved, q=x["q"])
    qe, ke, ve = expect(x, interleaved)
    assert np.array_equal(bits(q), qe) and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)
    assert pkv.get_last_error() == 0


@gpu
def test_write_rope_without_queries_in_place_and_into_a_given_buffer(pkvlib):
    x = inputs(40, 8, 2, 128, seed=5, strided=False)
    qe, ke, ve = expect(x, False)
    none, kc, vc = call(x, False)
    assert none is None and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)
    out = torch.empty_like(x["q"])
    q, _, _ = call(x, False, q=x["q"], q_out=out)
    assert q is out and np.array_equal(bits(out), qe)
    q, _, _ = call(x, False, q=x["q"], q_out=x["q"])  # in place, last: it overwrites the input
    assert np.array_equal(bits(x["q"]), qe)


@gpu
def test_write_rope_skips(pkvlib):
    """Negative slots and slots beyond the pool keep the queries and skip the
    pages; a position outside the table skips the token whole."""
    pkv.get_last_error()
    x = inputs(20, 8, 2, 64, seed=6)
    slots = x["slots"].copy()
    slots[[0, 7]] = -1
    q, kc, vc = call(x, True, slots=slots, q=x["q"])
    qe, ke, ve = expect(x, True, slots=slots)
    assert np.array_equal(bits(q), qe) and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)
    assert pkv.get_last_error() == 0
    beyond = slots.copy()
    beyond[3] = x["kc"].shape[0] * 16
    slots[3] = -1
    q, kc, vc = call(x, True, slots=beyond, q=x["q"])
    qe, ke, ve = expect(x, True, slots=slots)
    assert np.array_equal(bits(q), qe) and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)
    assert pkv.get_last_error() == pkv.STATUS_BAD_SLOT
    good = x["positions"].copy()
    out = torch.zeros(x["q"].shape, dtype=torch.bfloat16, device="cuda")
    x["positions"][[5, 6]] = [512, -1]
    q, kc, vc = call(x, True, slots=slots, q=x["q"], q_out=out)
    assert pkv.get_last_error() == pkv.STATUS_BAD_POSITION
    x["positions"] = good
    slots[[5, 6]] = -1
    qe, ke, ve = expect(x, True, slots=slots)
    qe[[5, 6]] = 0
    assert np.array_equal(bits(q), qe) and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,rot", [(1, 8, 2, 128), (33, 32, 8, 64), (700, 8, 8, 112)])
def test_write_rope_fp8_bits(pkvlib, T, hq, hkv, rot, interleaved):
    x = inputs(T, hq, hkv, rot, seed=T + 1)
    x["k"][0, 0] = 0  # a row of zeros takes the smallest scale
    x["v"][T // 2] *= 2.0 ** -100
    if T > 2:
        x["k"][1] *= 2.0 ** 90
    rng = np.random.default_rng(T)
    shape = x["kc"].shape
    codes = [rng.integers(0, 127, size=tuple(shape), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(100, 140, size=tuple(shape[:3]), dtype=np.uint8) for _ in range(2)]
    dev = [cuda(a) for a in codes + scales]
    slots = x["slots"].copy()
    slots[T // 3] = slots[T // 3] if T < 3 else -1
    q = pkv.write_rope_fp8(x["k"], x["v"], cuda(x["positions"]), cuda(x["table"]), cuda(slots), *dev, q=x["q"],
                           interleaved=interleaved)
    assert np.array_equal(bits(q), R.rotate_bits(bits(x["q"]), x["positions"], x["table"], interleaved))
    # V rows go through the 8-bit write; K rows are quantised from fp32
    _, vc, _, vs = write_fp8(bits(x["v"]), bits(x["v"]), slots, *codes, *scales, 16)
    kq, kqs = R.quantize_values(R.rotate(bf16_to_f64(bits(x["k"])), x["table"][x["positions"]], interleaved))
    kc, ks = codes[0].copy(), scales[0].copy()
    for t, s in enumerate(slots):
        if s >= 0:
            kc[s // 16, :, s % 16], ks[s // 16, :, s % 16] = kq[t], kqs[t]
    for got, want in zip(dev, (kc, vc, ks, vs)):
        assert np.array_equal(got.cpu().numpy(), want)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (5, 20), (64, 16), (1000, 3), (2600, 1)])
def test_write_latent_bits(pkvlib, T, H, interleaved):
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    pages = -(-T // 16) + 2
    kv_a, qp, q0, pool = normal(T, 576), normal(T, H, 192), normal(T, H, 576), normal(pages, 16, 576)
    positions, slots = rng.integers(0, 300, size=T), rng.permutation(pages * 16)[:T]
    if T > 3:
        slots[2] = -1
    tab = table(300, 64)
    out, cache = q0.clone(), pool.clone()
    got = pkv.write_latent(kv_a[:, :512], kv_a[:, 512:], cuda(positions), cuda(tab), cuda(slots), cache,
                           q_pe=qp[..., 128:], q_out=out, interleaved=interleaved)
    assert got is out
    want = bits(q0)
    want[..., 512:] = R.rotate_bits(bits(qp[..., 128:]), positions, tab, interleaved)
    assert np.array_equal(bits(out), want)
    c, k = bits(kv_a[:, :512]), bits(kv_a[:, 512:])
    assert np.array_equal(bits(cache), R.write_latent(c, k, positions, tab, slots, bits(pool), interleaved))
    cache = pool.clone()
    assert pkv.write_latent(kv_a[:, :512], kv_a[:, 512:], cuda(positions), cuda(tab), cuda(slots), cache,
                            interleaved=interleaved) is None
    assert np.array_equal(bits(cache), R.write_latent(c, k, positions, tab, slots, bits(pool), interleaved))
    # in place: the rotated part of q_out itself
    out = q0.clone()
    pkv.write_latent(kv_a[:, :512], kv_a[:, 512:], cuda(positions), cuda(tab), cuda(slots), cache, q_pe=out[..., 512:],
                     q_out=out, interleaved=interleaved)
    want = bits(q0)
    want[..., 512:] = R.rotate_bits(want[..., 512:], positions, tab, interleaved)
    assert np.array_equal(bits(out), want)


@gpu
def test_write_latent_skips(pkvlib):
    pkv.get_last_error()
    T, H = 6, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    c, k, qp, q0, pool = normal(T, 512), normal(T, 64), normal(T, H, 64), normal(T, H, 576), normal(2, 16, 576)
    positions, tab = np.array([0, 3, 64, -5, 7, 63]), table(64, 64)
    slots = np.array([4, 32, 9, 10, -1, 31])
    out, cache = q0.clone(), pool.clone()
    pkv.write_latent(c, k, cuda(positions), cuda(tab), cuda(slots), cache, q_pe=qp, q_out=out)
    assert pkv.get_last_error() == pkv.STATUS_BAD_SLOT | pkv.STATUS_BAD_POSITION
    ok = np.array([0, 1, 4, 5])
    want = bits(q0)
    want[ok, :, 512:] = R.rotate_bits(bits(qp)[ok], positions[ok], tab, False)
    assert np.array_equal(bits(out), want)
    kept = slots[ok].copy()
    kept[1] = -1
    assert np.array_equal(bits(cache), R.write_latent(bits(c)[ok], bits(k)[ok], positions[ok], tab, kept, bits(pool),
                                                      False))
