"""The compiled argument checks of the rotated appends and of latent
attention: every refusal is an exception before a launch, tensors made on the
way belong to the caller's stream, and other types of numbers are taken as
Python takes them."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv

gpu = pytest.mark.gpu
BF = torch.bfloat16


def rope_args(device="cuda", T=4, hq=8, hkv=2, **over):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=device)
    a = dict(k_new=z(T, hkv, 128), v_new=z(T, hkv, 128), positions=z(T, dt=torch.int64), cos_sin=z(8, 128, dt=torch.float32),
             slot_mapping=torch.arange(T, device=device), k_cache=z(4, hkv, 16, 128), v_cache=z(4, hkv, 16, 128),
             q=z(T, hq, 128))
    a.update(over)
    return a


def latent_write_args(device="cuda", T=4, H=3, **over):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=device)
    a = dict(c_new=z(T, 512), k_pe=z(T, 64), positions=z(T, dt=torch.int64), cos_sin=z(8, 64, dt=torch.float32),
             slot_mapping=torch.arange(T, device=device), latent_cache=z(4, 16, 576), q_pe=z(T, H, 64))
    a.update(over)
    return a


def attend_args(device="cuda", B=2, H=3, **over):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=device)
    a = dict(q=z(B, H, 576), latent_cache=z(4, 16, 576), block_tables=z(B, 2, dt=torch.int32),
             seq_lens=torch.ones(B, dtype=torch.int32, device=device),
             query_start_loc=torch.arange(B + 1, dtype=torch.int32, device=device), scale=0.1)
    a.update(over)
    return a


def test_the_compiled_checks_on_host_tensors(pkvlib):
    """Called past the package's own first check, as a library without a GPU
    can call them: types first, then the device, then the number of arguments."""
    n = pkv._native()
    a = rope_args("cpu")
    order = lambda a, *names: [a[k] for k in names]
    rope = ("k_new", "v_new", "positions", "cos_sin", "slot_mapping", "k_cache", "v_cache", "q")
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        n.write_rope(0, None, *order(a, *rope), None, False)
    with pytest.raises(TypeError, match="k_cache must be torch.bfloat16, got torch.float32"):
        n.write_rope(0, None, *order(rope_args("cpu", k_cache=torch.zeros(4, 2, 16, 128)), *rope), None, False)
    with pytest.raises(TypeError, match="k_cache must be torch.uint8, got torch.bfloat16"):
        n.write_rope_fp8(0, None, *order(a, *rope), None, False, None, None)
    with pytest.raises(TypeError, match="latent_cache must be a torch.Tensor"):
        n.write_latent(0, None, *[None] * 9)
    with pytest.raises(TypeError, match="latent_cache must be a torch.Tensor"):
        n.attend_latent(0, None, *[None] * 9)
    for call in (n.write_rope, n.write_rope_fp8, n.write_latent, n.attend_latent, n.bind):
        with pytest.raises(TypeError, match="arguments"):
            call(0)


@gpu
@pytest.mark.parametrize("bad,error,words", [
    (dict(k_new=[0.0]), TypeError, "k_new must be a torch.Tensor"),
    (dict(k_new=torch.zeros(4, 2, 128)), TypeError, "k_new must be torch.bfloat16"),
    (dict(k_new=torch.zeros(4, 2, 128, dtype=BF)), ValueError, "k_new must be a CUDA tensor"),
    (dict(v_new=lambda: torch.zeros(5, 2, 128, dtype=BF, device="cuda")), ValueError, "v_new must be"),
    (dict(v_new=lambda: torch.zeros(4, 128, 2, dtype=BF, device="cuda").transpose(1, 2)), ValueError, "contiguous"),
    (dict(k_new=lambda: torch.zeros(4, 260, dtype=BF, device="cuda")[:, :256].view(4, 2, 128)), ValueError, "stride"),
    (dict(k_new=lambda: torch.zeros(1, 2, 128, dtype=BF, device="cuda").expand(4, 2, 128)), ValueError, "stride"),
    (dict(positions=lambda: torch.zeros(4, dtype=torch.int32, device="cuda")), TypeError, "positions must be torch.int64"),
    (dict(positions=lambda: torch.zeros(8, dtype=torch.int64, device="cuda")[::2]), ValueError, "positions must be contig"),
    (dict(slot_mapping=lambda: torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError, "disagree"),
    (dict(cos_sin=lambda: torch.zeros(8, 2, 64, device="cuda")), ValueError, "cos_sin must be"),
    (dict(q=lambda: torch.zeros(4, 128, dtype=BF, device="cuda")), ValueError, "q must be"),
    (dict(q=lambda: torch.zeros(4, 0, 128, dtype=BF, device="cuda")), ValueError, "q must be"),
    (dict(q=None, q_out=lambda: torch.zeros(4, 8, 128, dtype=BF, device="cuda")), ValueError, "q_out without q"),
    (dict(q_out=lambda: torch.zeros(4, 4, 128, dtype=BF, device="cuda")), ValueError, "q_out"),
    (dict(v_cache=lambda: torch.zeros(5, 2, 16, 128, dtype=BF, device="cuda")), ValueError, "disagree"),
    (dict(k_cache=lambda: torch.zeros(4, 2, 16, 256, dtype=BF, device="cuda")[..., :128]), ValueError, "contiguous"),
    (dict(cos_sin=lambda: torch.zeros(8, 120, device="cuda")), pkv.PkvError, "pkv_write_rope"),
    (dict(stream="s"), AttributeError, "cuda_stream"),
])
def test_write_rope_refuses_before_a_launch(pkvlib, bad, error, words):
    bad = {k: v() if callable(v) else v for k, v in bad.items()}
    before = pkv.launch_count()
    with pytest.raises(error, match=words):
        pkv.write_rope(**rope_args(**bad))
    assert pkv.launch_count() == before


@gpu
@pytest.mark.parametrize("bad,error,words", [
    (dict(c_new=lambda: torch.zeros(4, 576, dtype=BF, device="cuda")), ValueError, "c_new must be"),
    (dict(k_pe=lambda: torch.zeros(4, 1, 64, dtype=BF, device="cuda")), ValueError, "k_pe must be"),
    (dict(q_pe=lambda: torch.zeros(4, 3, 128, dtype=BF, device="cuda")), ValueError, "q_pe must be"),
    (dict(q_pe=lambda: torch.zeros(4, 1, 64, dtype=BF, device="cuda").expand(4, 3, 64)), ValueError, "strides"),
    (dict(q_pe=lambda: torch.zeros(4, 3, 68, dtype=BF, device="cuda")[..., :64]), ValueError, "strides"),
    (dict(q_out=lambda: torch.zeros(4, 3, 512, dtype=BF, device="cuda")), ValueError, "q_out must be"),
    (dict(q_pe=None, q_out=lambda: torch.zeros(4, 3, 576, dtype=BF, device="cuda")), ValueError, "q_out without"),
    (dict(cos_sin=lambda: torch.zeros(8, 32, device="cuda")), pkv.PkvError, "pkv_write_latent"),
    (dict(latent_cache=lambda: torch.zeros(4, 16, 512, dtype=BF, device="cuda")), pkv.PkvError, "pkv_write_latent"),
])
def test_write_latent_refuses_before_a_launch(pkvlib, bad, error, words):
    bad = {k: v() if callable(v) else v for k, v in bad.items()}
    before = pkv.launch_count()
    with pytest.raises(error, match=words):
        pkv.write_latent(**latent_write_args(**bad))
    assert pkv.launch_count() == before


@gpu
@pytest.mark.parametrize("bad,error,words", [
    (dict(q=lambda: torch.zeros(2, 3, 512, dtype=BF, device="cuda")), ValueError, "rows disagree"),
    (dict(q=lambda: torch.zeros(3, 2, 576, dtype=BF, device="cuda").transpose(0, 1)), ValueError, "q must be contiguous"),
    (dict(block_tables=lambda: torch.zeros(3, 2, dtype=torch.int32, device="cuda")), ValueError, "disagree"),
    (dict(seq_lens=lambda: torch.ones(2, dtype=torch.int64, device="cuda")), TypeError, "seq_lens must be torch.int32"),
    (dict(query_start_loc=lambda: torch.zeros(2, dtype=torch.int32, device="cuda")), ValueError, "disagree"),
    (dict(out=lambda: torch.zeros(2, 3, 576, dtype=BF, device="cuda")), ValueError, "out must be"),
    (dict(out=lambda: torch.zeros(2, 3, 512, device="cuda")), TypeError, "out must be torch.bfloat16"),
    (dict(workspace=lambda: torch.zeros(256, dtype=torch.uint8, device="cuda")), pkv.PkvError, "pkv_attend_latent"),
    (dict(scale=None), TypeError, "float"),
    (dict(max_query_len="x"), ValueError, "int"),
    (dict(q=lambda: torch.zeros(2, 257, 576, dtype=BF, device="cuda")), pkv.PkvError, "pkv_attend_latent"),
])
def test_attend_latent_refuses_before_a_launch(pkvlib, bad, error, words):
    bad = {k: v() if callable(v) else v for k, v in bad.items()}
    before = pkv.launch_count()
    with pytest.raises(error, match=words):
        pkv.attend_latent(**attend_args(**bad))
    assert pkv.launch_count() == before


@gpu
def test_numbers_streams_and_empty_calls(pkvlib):
    pkv.get_last_error()
    a = attend_args()
    a["latent_cache"].normal_()
    a["q"].normal_()
    want = pkv.attend_latent(**a)
    for more in (dict(scale=np.float32(0.1)), dict(scale=np.float64(0.1)), dict(max_query_len=np.int64(1)),
                 dict(max_query_len=1 << 70), dict(max_query_len=-(1 << 70)), dict(max_query_len=1.0)):
        got = pkv.attend_latent(**{**a, **more})
        torch.testing.assert_close(got.float(), want.float(), rtol=2**-7, atol=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.attend_latent(**a, stream=side)  # out and workspace made on that stream
    q = pkv.write_rope(**rope_args(), stream=side)
    side.synchronize()
    assert torch.equal(got, want) and q.shape == (4, 8, 128) and not bool(q.any())
    before = pkv.launch_count()
    none = rope_args(T=0)
    assert pkv.write_rope(**none).shape == (0, 8, 128)
    assert pkv.write_latent(**latent_write_args(T=0)).shape == (0, 3, 576)
    assert pkv.attend_latent(**attend_args(B=0)).shape == (0, 3, 512)
    assert pkv.launch_count() == before
    # what is returned is the tensor that was given, and inputs that need a gradient are read like others
    out = torch.empty(2, 3, 512, dtype=BF, device="cuda")
    refs = __import__("sys").getrefcount(out)
    for _ in range(5):
        assert pkv.attend_latent(**{**a, "q": a["q"].detach().requires_grad_()}, out=out) is out
    assert __import__("sys").getrefcount(out) == refs and torch.equal(out, want)
    assert pkv.get_last_error() == 0
