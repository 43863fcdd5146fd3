"""Calls behind one another on a stream, where the next one's kernel is let in
before the last one's has ended: pkv_attend stamps counters in its workspace.
That memory may be what the call before has just been given as inputs or
scratch and no longer needs: a stream's order is all a caller owes it."""

import numpy as np
import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from helpers import bits
from oracle import rotary_latent as R
from oracle.pkv_oracle import write
from test_latent import WIDE, Case, cuda
from test_rope import table

pytestmark = pytest.mark.gpu


class Stamper:
    """A pkv_attend call whose counters fill ``size`` bytes at the start of the
    workspace that it is given: 8 bytes a (token, kv head)."""

    def __init__(self, size, hkv=32, seqs=64):
        T = -(-size // (8 * hkv))
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
        n = np.minimum(8, np.maximum(0, T - 8 * np.arange(seqs)))  # (rows behind the last sequence are stamped too)
        qsl = np.concatenate([[0], np.cumsum(n)])
        self.args = (normal(T, hkv, 128), normal(4, hkv, 16, 128), normal(4, hkv, 16, 128),
                     cuda(np.tile(np.arange(4, dtype=np.int32), (seqs, 1))), cuda(np.full(seqs, 50, np.int32)),
                     cuda(qsl, np.int32), 0.088)
        self.out = torch.empty(T, hkv, 128, device="cuda", dtype=torch.bfloat16)
        desc = pkv.make_desc(self.args[1], hkv, 4)
        self.need = pkv.workspace_size(desc, seqs, T)
        self.rows = int(qsl[-1])
        self.want = pkv.attend(*self.args, max_query_len=8)

    def __call__(self, buf):
        assert buf.numel() >= self.need
        pkv.attend(*self.args, out=self.out, workspace=buf, max_query_len=8)

    def check(self):
        torch.testing.assert_close(self.out[:self.rows].float(), self.want[:self.rows].float(), rtol=2**-7, atol=1e-2)


@pytest.mark.parametrize("lens,H,width", [([3000, 200, 77], 20, 1), ([9000], 3, 1), ([3000, 900, 77], 96, WIDE),
                                          ([700] * 100, 70, WIDE), ([70, 200, 77], 16, 1)])
def test_counters_over_partials_and_join_records(pkvlib, lens, H, width):
    """Over the partials at the workspace's start, and over the join records at
    its end, while the joining kernel's blocks end one by one: cut tiles of few
    rows leave most of a block's warps without work."""
    pkv.get_last_error()
    c = Case(lens, [1] * len(lens), H, seed=41, width=width)
    args = c.args()
    want = pkv.attend_latent(*args, max_query_len=1)
    c.check(want)
    stamp = Stamper(4 << 20)
    size = pkv.workspace_size_latent(pkv.make_latent_desc(c.pool, H, c.tables.shape[1]), len(lens), len(lens))
    buf = torch.full((size + stamp.need,), 255, device="cuda", dtype=torch.uint8)
    tail = (size - 4096) // 256 * 256
    got = []
    for i in range(40):
        got.append(pkv.attend_latent(*args, workspace=buf[:size], max_query_len=1))
        stamp(buf if i & 1 else buf[tail:])
    torch.cuda.synchronize()
    assert all(torch.equal(g.view(torch.int16), want.view(torch.int16)) for g in got)
    stamp.check()
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("T,hq,hkv", [(3, 32, 8), (300, 4, 4), (4001, 8, 2)])
def test_counters_over_the_inputs_of_a_rotated_append(pkvlib, T, hq, hkv):
    """The projection's memory is the next call's workspace; every other token
    is padding, whose warps are done early."""
    pkv.get_last_error()
    stamp = Stamper(T * (hq + 2 * hkv) * 256)
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    pages = -(-T // 16) + 1
    src, pos, slots = normal(T, hq + 2 * hkv, 128), rng.integers(0, 300, T), rng.permutation(pages * 16)[:T]
    slots[::2] = -1
    tab = table(300, 128)
    buf = torch.zeros(max(stamp.need, src.numel() * 2), dtype=torch.uint8, device="cuda")
    qkv = buf[:src.numel() * 2].view(torch.bfloat16).view(src.shape)
    kc, vc = normal(pages, hkv, 16, 128), normal(pages, hkv, 16, 128)
    want_q = R.rotate_bits(bits(src[:, :hq]), pos, tab, False)
    want_k, want_v = write(R.rotate_bits(bits(src[:, hq:hq + hkv]), pos, tab, False), bits(src[:, hq + hkv:]), slots,
                           bits(kc), bits(vc), 16)
    meta, q_out = (cuda(pos), cuda(tab), cuda(slots)), torch.empty(T, hq, 128, device="cuda", dtype=torch.bfloat16)
    for _ in range(20):
        qkv.copy_(src)
        k, v = kc.clone(), vc.clone()
        pkv.write_rope(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *meta, k, v, q=qkv[:, :hq], q_out=q_out)
        stamp(buf)
        assert np.array_equal(bits(q_out), want_q)
        assert np.array_equal(bits(k), want_k) and np.array_equal(bits(v), want_v)
    stamp.check()
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("T,H", [(5, 128), (600, 3), (3001, 1)])
def test_counters_over_the_inputs_of_a_latent_append(pkvlib, T, H):
    pkv.get_last_error()
    stamp = Stamper(T * 576 * 2)
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    pages = -(-T // 16) + 1
    src, qp, q0, pool = normal(T, 576), normal(T, H, 64), normal(T, H, 576), normal(pages, 16, 576)
    pos, slots, tab = rng.integers(0, 300, T), rng.permutation(pages * 16)[:T], table(300, 64)
    slots[1::2] = -1
    buf = torch.zeros(max(stamp.need, src.numel() * 2), dtype=torch.uint8, device="cuda")
    kv = buf[:src.numel() * 2].view(torch.bfloat16).view(src.shape)
    want = R.write_latent(bits(src[:, :512]), bits(src[:, 512:]), pos, tab, slots, bits(pool), True)
    want_q = bits(q0)
    want_q[..., 512:] = R.rotate_bits(bits(qp), pos, tab, True)
    meta = cuda(pos), cuda(tab), cuda(slots)
    for _ in range(20):
        kv.copy_(src)
        cache, q = pool.clone(), q0.clone()
        pkv.write_latent(kv[:, :512], kv[:, 512:], *meta, cache, q_pe=qp, q_out=q, interleaved=True)
        stamp(buf)
        assert np.array_equal(bits(cache), want) and np.array_equal(bits(q), want_q)
    stamp.check()
    assert pkv.get_last_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,hkv", [(64, 8), (4001, 8), (9001, 2)])
def test_counters_over_the_inputs_of_a_plain_append(pkvlib, T, hkv, fp8):
    """pkv_write and pkv_write_fp8 let the next kernel in as they start."""
    pkv.get_last_error()
    stamp = Stamper(2 * T * hkv * 256)
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    pages = -(-T // 16) + 1
    src = torch.randn(2, T, hkv, 128, generator=gen, device="cuda").to(torch.bfloat16)
    slots = cuda(rng.permutation(pages * 16)[:T])
    buf = torch.zeros(max(stamp.need, src.numel() * 2), dtype=torch.uint8, device="cuda")
    k, v = buf[:src.numel() * 2].view(torch.bfloat16).view(src.shape)
    kind = torch.uint8 if fp8 else torch.bfloat16
    shapes = [(pages, hkv, 16, 128)] * 2 + [(pages, hkv, 16)] * (2 * fp8)
    append = pkv.write_fp8 if fp8 else pkv.write
    want = [torch.zeros(s, dtype=kind, device="cuda") for s in shapes]
    append(src[0], src[1], slots, *want)
    torch.cuda.synchronize()
    for _ in range(20):
        k.copy_(src[0])
        v.copy_(src[1])
        pools = [torch.zeros(s, dtype=kind, device="cuda") for s in shapes]
        append(k, v, slots, *pools)
        stamp(buf)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pools, want))
    stamp.check()
    assert pkv.get_last_error() == 0
