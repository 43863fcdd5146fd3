"""Refusals of the rotated appends and of latent attention, all on the host,
and the NumPy forms they are tested against."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from oracle import rotary_latent as R

FAKE = 1 << 20  # 16-byte aligned, never dereferenced
NULL, SHAPE, ALIGN, RANGE = -1, -3, -2, -4


def _desc(**kw):
    d = dict(num_blocks=64, page_size=16, num_kv_heads=2, num_q_heads=8, head_dim=128, max_blocks_per_seq=16)
    d.update(kw)
    return pkv.Desc(**d)


def _latent(**kw):
    return _desc(**{**dict(num_kv_heads=1, num_q_heads=20, head_dim=576), **kw})


def _rope(lib, desc=None, fp8=False, rot=128, max_pos=64, table=FAKE, T=4, qs=1024, ks=256, vs=256, **ptr):
    p = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, slots=FAKE, q_out=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE)
    p.update(ptr)
    rope = pkv.Rope(table, max_pos, rot, 0)
    pools = [p["kc"], p["vc"]] + ([p["ksc"], p["vsc"]] if fp8 else [])
    fn = lib.pkv_write_rope_fp8 if fp8 else lib.pkv_write_rope
    return fn(p["q"], p["k"], p["v"], qs, ks, vs, p["pos"], p["slots"], T, ctypes.byref(rope), p["q_out"], *pools,
              ctypes.byref(desc or _desc()), None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(rot=24), SHAPE), (dict(rot=0), SHAPE), (dict(rot=144), SHAPE), (dict(max_pos=0), RANGE),
    (dict(table=None), NULL), (dict(table=FAKE + 8), ALIGN), (dict(T=-1), RANGE), (dict(ks=248), SHAPE),
    (dict(vs=260), SHAPE), (dict(qs=1016), SHAPE), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(k=FAKE + 2), ALIGN), (dict(q_out=FAKE + 8), ALIGN),
    (dict(pos=FAKE + 4), ALIGN), (dict(kc=None), NULL), (dict(desc=_desc(head_dim=64)), SHAPE),
])
def test_write_rope_refuses(pkvlib, fp8, bad, code):
    before = pkvlib.pkv_launch_count()
    assert _rope(pkvlib, fp8=fp8, **bad) == code
    assert _rope(pkvlib, fp8=fp8, T=0) == 0
    assert pkvlib.pkv_launch_count() == before


def test_write_rope_fp8_needs_scales(pkvlib):
    assert _rope(pkvlib, fp8=True, ksc=None) == NULL
    assert _rope(pkvlib, fp8=True, vsc=FAKE + 4) == ALIGN


def _write_latent(lib, desc=None, rot=64, T=4, cs=512, ks=64, qs=1280, hs=64, **ptr):
    p = dict(c=FAKE, k=FAKE, q=FAKE, pos=FAKE, slots=FAKE, q_out=FAKE, pool=FAKE)
    p.update(ptr)
    rope = pkv.Rope(FAKE, 64, rot, 0)
    return lib.pkv_write_latent(p["c"], p["k"], p["q"], cs, ks, qs, hs, p["pos"], p["slots"], T, ctypes.byref(rope),
                                p["q_out"], p["pool"], ctypes.byref(desc or _latent()), None)


@pytest.mark.parametrize("bad,code", [
    (dict(rot=32), SHAPE), (dict(rot=128), SHAPE), (dict(cs=504), SHAPE), (dict(ks=60), SHAPE), (dict(hs=56), SHAPE),
    (dict(qs=1272), SHAPE), (dict(c=None), NULL), (dict(q=None), NULL), (dict(pool=FAKE + 8), ALIGN), (dict(T=-2), RANGE),
    (dict(desc=_latent(head_dim=512)), SHAPE), (dict(desc=_latent(num_kv_heads=2)), SHAPE),
    (dict(desc=_latent(num_q_heads=257)), SHAPE), (dict(desc=_latent(page_size=64)), SHAPE),
    (dict(desc=_latent(num_blocks=0)), RANGE),
])
def test_write_latent_refuses(pkvlib, bad, code):
    assert _write_latent(pkvlib, **bad) == code
    assert _write_latent(pkvlib, T=0) == 0


def _attend(lib, desc=None, B=4, T=4, **ptr):
    p = dict(q=FAKE, pool=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, out=FAKE, ws=FAKE)
    p.update(ptr)
    return lib.pkv_attend_latent(p["q"], p["pool"], p["bt"], p["sl"], p["qsl"], B, T, 0, 0.1, p["out"], p["ws"],
                                 1 << 30, ctypes.byref(desc or _latent()), None)


@pytest.mark.parametrize("bad,code", [
    (dict(desc=_latent(head_dim=128)), SHAPE), (dict(desc=_latent(num_q_heads=0)), SHAPE), (dict(B=2049), RANGE),
    (dict(B=-1), RANGE), (dict(T=-1), RANGE), (dict(q=None), NULL), (dict(ws=None), NULL), (dict(bt=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(ws=FAKE + 128), ALIGN), (dict(sl=FAKE + 2), ALIGN), (dict(out=FAKE + 4), ALIGN),
])
def test_attend_latent_refuses(pkvlib, bad, code):
    before = pkvlib.pkv_launch_count()
    assert _attend(pkvlib, **bad) == code
    assert _attend(pkvlib, B=0) == 0 and _attend(pkvlib, T=0) == 0
    n = ctypes.c_size_t(0)
    if set(bad) <= {"desc", "B", "T"}:
        assert pkvlib.pkv_attend_latent_workspace_size(ctypes.byref(bad.get("desc", _latent())), bad.get("B", 4),
                                                       bad.get("T", 4), ctypes.byref(n)) == code
    assert pkvlib.pkv_launch_count() == before


@pytest.mark.parametrize("bad", [
    dict(desc=_latent(num_q_heads=256), T=2**23), dict(desc=_latent(num_blocks=2**30)),
    dict(desc=_latent(max_blocks_per_seq=2**27 - 64)), dict(desc=_latent(max_blocks_per_seq=2**31 - 1)),
    dict(desc=_latent(num_q_heads=256, max_blocks_per_seq=2**27 - 65), T=2**22),
])
def test_attend_latent_refuses_what_leaves_its_integers(pkvlib, bad):
    assert _attend(pkvlib, **bad) == RANGE


def test_binding_refuses_types_and_host_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64)
    tab = torch.zeros(8, 128)
    with pytest.raises(TypeError, match="k_cache"):
        pkv.write_rope(bf(4, 2, 128), bf(4, 2, 128), ids, tab, ids, [0.0], bf(8, 2, 16, 128))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.write_rope(bf(4, 2, 128), bf(4, 2, 128), ids, tab, ids, bf(8, 2, 16, 128), bf(8, 2, 16, 128))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.write_latent(bf(4, 512), bf(4, 64), ids, tab[:, :64], ids, bf(8, 16, 576))
    with pytest.raises(TypeError, match="latent_cache must be"):
        pkv.attend_latent(bf(4, 8, 576), None, ids, ids, ids, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.attend_latent(bf(4, 8, 576), bf(8, 16, 576), ids, ids, ids, 0.1)


# ---- the NumPy forms ----------------------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64)).astype(np.float32).astype(np.float64)
    angle = rng.uniform(-9, 9, (5, 16))
    tab = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
    got = R.rotate(x, tab, interleaved)
    pairs = x[..., :32].reshape(5, 3, 16, 2) if interleaved else np.stack([x[..., :16], x[..., 16:32]], -1)
    z = (pairs[..., 0] + 1j * pairs[..., 1]) * np.exp(1j * angle)[:, None]
    back = np.stack([z.real, z.imag], -1)
    want = back.reshape(5, 3, 32) if interleaved else np.concatenate([back[..., 0], back[..., 1]], -1)
    # two products, a sum and the table's own rounding, each within 2^-24 of magnitudes up to |z|
    assert np.abs(got[..., :32] - want).max() <= 4 * 2.0 ** -24 * np.abs(z).max() * 2
    assert np.array_equal(got[..., 32:], x[..., 32:])


def test_latent_attention_form():
    """One key gives its value; equal keys give the mean of the values seen."""
    rng = np.random.default_rng(1)
    to_bits = lambda x: R.f64_to_bf16(x)
    pool = rng.standard_normal((3, 16, 576))
    pool_bits = to_bits(pool)
    q = to_bits(rng.standard_normal((2, 4, 576)))
    one, _ = R.attend_latent(q[:1], pool_bits, [[2]], [1], [0, 1], 0.1)
    assert np.allclose(one[0], np.broadcast_to(R.bf16_to_f64(pool_bits[2, 0, :512]), (4, 512)), atol=1e-12)
    out, _ = R.attend_latent(np.zeros_like(q), pool_bits, [[1, 0]], [20], [0, 2], 0.1)
    rows = R.bf16_to_f64(np.concatenate([pool_bits[1], pool_bits[0]]))[:, :512]
    assert np.allclose(out[0, 0], rows[:19].mean(0)) and np.allclose(out[1, 3], rows[:20].mean(0))
