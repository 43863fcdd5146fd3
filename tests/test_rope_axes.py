"""Appends of tokens with several positions: bit for bit against the NumPy
form (the rotation is defined in fp32 arithmetic and rounded once), and
against write_rope where all axes agree."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits
from oracle import rotary_latent as R
from oracle.pkv_oracle import bf16_to_f64, write, write_fp8
from test_rope import cuda, inputs, table

gpu = pytest.mark.gpu
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
NULL, ALIGN, SHAPE, RANGE = -1, -2, -3, -4


def rows_of(tab, positions, axes):
    """[T, R]: for each token its cosines and sines, pair by pair from the row of the pair's axis."""
    half = tab.shape[1] // 2
    out = np.empty((positions.shape[1], 2 * half), np.float32)
    for i, a in enumerate(axes):
        out[:, i] = tab[positions[a], i]
        out[:, half + i] = tab[positions[a], half + i]
    return out


def layouts(half, A):
    first = half // (A + 1)
    return {"blocks": [0] * first + [1 + i * (A - 1) // (half - first) if A > 1 else 0 for i in range(half - first)],
            "in turn": [i % A for i in range(half)],
            "any": np.random.default_rng(half + A).integers(0, A, size=half).tolist()}


def several(x, A, seed):
    """Positions [A, T] for the tokens of inputs()."""
    return np.random.default_rng(seed).integers(0, x["table"].shape[0], size=(A, len(x["slots"])))


# ---- host -----------------------------------------------------------------------


def test_rope_axes_names_the_axis_of_every_pair():
    assert pkv.rope_axes((2, 3, 1)) == bytes([0, 0, 1, 1, 1, 2])
    assert pkv.rope_axes((2, 3, 1), in_turn=True) == bytes([0, 1, 2, 0, 1, 1])
    assert pkv.rope_axes((0, 4)) == bytes([1] * 4)
    for bad in ((), (3, -1)):
        with pytest.raises(ValueError):
            pkv.rope_axes(bad)


def _call(lib, fp8=False, desc=None, rot=128, max_pos=64, tab=FAKE, A=3, axes=None, stride=4, T=4, qs=1024, ks=256,
          vs=256, rope=True, **ptr):
    p = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, slots=FAKE, q_out=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE)
    p.update(ptr)
    axes = (ctypes.c_uint8 * 64)(*(axes if axes is not None else [i % 3 for i in range(64)]))
    r = pkv.RopeAxes(tab, max_pos, rot, 0, A, ctypes.addressof(axes) if p.get("axis_of", 1) else None)
    d = desc or pkv.Desc(64, 16, 2, 8, 128, 16)
    pools = [p["kc"], p["vc"]] + ([p["ksc"], p["vsc"]] if fp8 else [])
    fn = lib.pkv_write_rope_axes_fp8 if fp8 else lib.pkv_write_rope_axes
    return fn(p["q"], p["k"], p["v"], qs, ks, vs, p["pos"], stride, p["slots"], T, ctypes.byref(r) if rope else None,
              p["q_out"], *pools, ctypes.byref(d), None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(A=0), RANGE), (dict(A=5), RANGE), (dict(A=2), RANGE), (dict(stride=-1), RANGE), (dict(axis_of=None), NULL),
    (dict(rope=False), NULL), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(max_pos=0), RANGE),
    (dict(tab=FAKE + 8), ALIGN), (dict(T=-1), RANGE), (dict(ks=248), SHAPE), (dict(q=None), NULL),
    (dict(pos=None), NULL), (dict(pos=FAKE + 4), ALIGN), (dict(desc=pkv.Desc(64, 16, 2, 8, 64, 16)), SHAPE),
])
def test_write_rope_axes_refuses(pkvlib, fp8, bad, code):
    before = pkvlib.pkv_launch_count()
    assert _call(pkvlib, fp8=fp8, **bad) == code
    assert _call(pkvlib, fp8=fp8, T=0) == 0 and _call(pkvlib, fp8=fp8, T=0, rope=False) == 0
    assert pkvlib.pkv_launch_count() == before


def test_axes_behind_the_rotated_pairs_are_not_read(pkvlib):
    """rotary_dim 32 has 16 pairs: what stands behind them may be anything (refused for its device, not its axes)."""
    axes = [i % 3 for i in range(16)] + [200] * 48
    assert _call(pkvlib, rot=32, axes=axes, ks=248) == SHAPE


# ---- GPU ------------------------------------------------------------------------


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["blocks", "in turn", "any"])
@pytest.mark.parametrize("T,hq,hkv,rot,A", [(1, 32, 8, 128, 3), (1, 1, 1, 16, 2), (3, 8, 8, 64, 4), (17, 16, 1, 96, 3),
                                            (129, 32, 2, 48, 1), (1120, 8, 2, 128, 3), (2500, 4, 4, 32, 2)])
def test_write_rope_axes_bits(pkvlib, T, hq, hkv, rot, A, layout, interleaved):
    x = inputs(T, hq, hkv, rot, seed=T + rot)
    axes, pos = layouts(rot // 2, A)[layout], several(x, A, T)
    if T > 3:
        x["slots"][2] = -1  # padding: no row, but its queries are turned
    kc, vc = x["kc"].clone(), x["vc"].clone()
    q = pkv.write_rope_axes(x["k"], x["v"], cuda(pos), bytes(axes), cuda(x["table"]), cuda(x["slots"]), kc, vc,
                            q=x["q"], interleaved=interleaved)
    rows = rows_of(x["table"], pos, axes)
    turn = lambda b: R.f64_to_bf16(R.rotate(bf16_to_f64(b), rows, interleaved))
    ke, ve = write(turn(bits(x["k"])), bits(x["v"]), x["slots"], bits(x["kc"]), bits(x["vc"]), 16)
    assert np.array_equal(bits(q), turn(bits(x["q"])))
    assert np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)
    assert pkv.get_last_error() == 0


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,rot,A", [(1, 8, 2, 128, 3), (33, 32, 8, 64, 4), (700, 8, 8, 112, 3)])
def test_write_rope_axes_fp8_bits(pkvlib, T, hq, hkv, rot, A, interleaved):
    x = inputs(T, hq, hkv, rot, seed=T + 1)
    x["k"][0, 0] = 0  # a row of zeros takes the smallest scale
    if T > 2:
        x["k"][1] *= 2.0 ** 90
    axes, pos = layouts(rot // 2, A)["in turn"], several(x, A, T)
    rng = np.random.default_rng(T)
    shape = x["kc"].shape
    codes = [rng.integers(0, 127, size=tuple(shape), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(100, 140, size=tuple(shape[:3]), dtype=np.uint8) for _ in range(2)]
    dev = [cuda(a) for a in codes + scales]
    q = pkv.write_rope_axes_fp8(x["k"], x["v"], cuda(pos), axes, cuda(x["table"]), cuda(x["slots"]), *dev, q=x["q"],
                                interleaved=interleaved)
    rows = rows_of(x["table"], pos, axes)
    assert np.array_equal(bits(q), R.f64_to_bf16(R.rotate(bf16_to_f64(bits(x["q"])), rows, interleaved)))
    _, vc, _, vs = write_fp8(bits(x["v"]), bits(x["v"]), x["slots"], *codes, *scales, 16)
    kq, kqs = R.quantize_values(R.rotate(bf16_to_f64(bits(x["k"])), rows, interleaved))
    kc, ks = codes[0].copy(), scales[0].copy()
    for t, s in enumerate(x["slots"]):
        kc[s // 16, :, s % 16], ks[s // 16, :, s % 16] = kq[t], kqs[t]
    for got, want in zip(dev, (kc, vc, ks, vs)):
        assert np.array_equal(got.cpu().numpy(), want)


@gpu
def test_axes_that_agree_are_write_rope(pkvlib):
    """Equal positions on all axes (text tokens), as an expanded row, as a slice
    of a longer buffer and as one axis: write_rope's bits."""
    x = inputs(77, 16, 4, 128, seed=3)
    one = cuda(x["positions"])
    kc, vc = x["kc"].clone(), x["vc"].clone()
    want = pkv.write_rope(x["k"], x["v"], one, cuda(x["table"]), cuda(x["slots"]), kc, vc, q=x["q"])
    buffer = torch.full((3, 100), -7, dtype=torch.int64, device="cuda")
    buffer[:, 11:88] = one
    axes = pkv.rope_axes((16, 24, 24))
    for positions, ax in ((one.expand(3, -1), axes), (buffer[:, 11:88], pkv.rope_axes((24, 20, 20), in_turn=True)),
                          (one[None], bytes(64))):
        k2, v2 = x["kc"].clone(), x["vc"].clone()
        got = pkv.write_rope_axes(x["k"], x["v"], positions, ax, cuda(x["table"]), cuda(x["slots"]), k2, v2, q=x["q"])
        assert torch.equal(got, want) and torch.equal(k2, kc) and torch.equal(v2, vc)
    assert pkv.get_last_error() == 0


@gpu
def test_write_rope_axes_skips(pkvlib):
    """A position outside the table on any axis skips the token whole."""
    pkv.get_last_error()
    x = inputs(20, 8, 2, 64, seed=6)
    axes, pos = layouts(32, 3)["blocks"], several(x, 3, 6)
    good = pos.copy()
    pos[0, 5], pos[1, 6], pos[2, 7] = 512, -1, 1 << 40
    slots = x["slots"].copy()
    slots[3] = x["kc"].shape[0] * 16  # beyond the pool: flagged, its queries turned
    out = torch.zeros(x["q"].shape, dtype=torch.bfloat16, device="cuda")
    kc, vc = x["kc"].clone(), x["vc"].clone()
    pkv.write_rope_axes(x["k"], x["v"], cuda(pos), axes, cuda(x["table"]), cuda(slots), kc, vc, q=x["q"], q_out=out)
    assert pkv.get_last_error() == pkv.STATUS_BAD_POSITION | pkv.STATUS_BAD_SLOT
    slots[[3, 5, 6, 7]] = -1
    rows = rows_of(x["table"], good, axes)
    turn = lambda b: R.f64_to_bf16(R.rotate(bf16_to_f64(b), rows, False))
    qe = turn(bits(x["q"]))
    qe[[5, 6, 7]] = 0
    ke, ve = write(turn(bits(x["k"])), bits(x["v"]), slots, bits(x["kc"]), bits(x["vc"]), 16)
    assert np.array_equal(bits(out), qe) and np.array_equal(bits(kc), ke) and np.array_equal(bits(vc), ve)


@gpu
def test_write_rope_axes_arguments(pkvlib):
    x = inputs(5, 8, 2, 64, seed=8)
    pos, tab, slots = cuda(several(x, 3, 8)), cuda(x["table"]), cuda(x["slots"])
    ok = dict(k_new=x["k"], v_new=x["v"], positions=pos, axes=bytes(32), cos_sin=tab, slot_mapping=slots,
              k_cache=x["kc"], v_cache=x["vc"])
    for error, bad in [(TypeError, dict(axes=3)), (TypeError, dict(axes=None)), (ValueError, dict(axes=bytes(31))),
                       (ValueError, dict(axes=[3] * 32)), (ValueError, dict(axes=[-1] * 32)),
                       (TypeError, dict(axes=["x"] * 32)), (ValueError, dict(positions=pos[0])),
                       (ValueError, dict(positions=pos[:, :4])), (TypeError, dict(positions=pos.int())),
                       (ValueError, dict(positions=pos.cpu())), (ValueError, dict(positions=pos.repeat(2, 1))),
                       (ValueError, dict(positions=pos.t().contiguous().t())), (ValueError, dict(positions=pos[:0]))]:
        with pytest.raises(error):
            pkv.write_rope_axes(**{**ok, **bad})
    assert pkv.write_rope_axes(**ok) is None


@gpu
def test_write_rope_axes_in_a_graph_on_another_stream(pkvlib):
    """Captured once, replayed with other positions in the same buffer."""
    x = inputs(9, 8, 2, 128, seed=10)
    axes = layouts(64, 3)["in turn"]
    pos, tab, slots = cuda(several(x, 3, 1)), cuda(x["table"]), cuda(x["slots"])
    kc, vc, out = x["kc"].clone(), x["vc"].clone(), torch.empty(x["q"].shape, dtype=torch.bfloat16, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        pkv.write_rope_axes(x["k"], x["v"], pos, axes, tab, slots, kc, vc, q=x["q"], q_out=out)
    fresh = several(x, 3, 2)
    pos.copy_(cuda(fresh))
    graph.replay()
    torch.cuda.synchronize()
    rows = rows_of(x["table"], fresh, axes)
    turn = lambda b: R.f64_to_bf16(R.rotate(bf16_to_f64(b), rows, False))
    ke, _ = write(turn(bits(x["k"])), bits(x["v"]), x["slots"], bits(x["kc"]), bits(x["vc"]), 16)
    assert np.array_equal(bits(out), turn(bits(x["q"]))) and np.array_equal(bits(kc), ke)
