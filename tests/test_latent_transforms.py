"""Tensors without memory of their own (those inside torch.func.vmap) are
refused by an exception, wherever they stand in a call's arguments."""

import pytest
import torch

import paged_kv_cache_pkv_gb300 as pkv
from test_latent_binding import attend_args, latent_write_args, rope_args

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call,make,names", [
    (pkv.write_rope, rope_args, ("k_new", "v_new", "positions", "cos_sin", "slot_mapping", "k_cache", "v_cache", "q")),
    (pkv.write_latent, latent_write_args, ("c_new", "k_pe", "positions", "cos_sin", "slot_mapping", "latent_cache", "q_pe")),
    (pkv.attend_latent, attend_args, ("q", "latent_cache", "block_tables", "seq_lens", "query_start_loc")),
])
def test_batched_tensors_are_refused(pkvlib, call, make, names):
    before = pkv.launch_count()
    for name in names:
        args = make()
        both = torch.stack([args[name]] * 2)
        with pytest.raises(RuntimeError, match="storage"):
            torch.func.vmap(lambda x: call(**{**args, name: x}))(both)
    assert pkv.launch_count() == before
    call(**make())  # and the interpreter goes on
    torch.cuda.synchronize()
    assert pkv.get_last_error() == 0
