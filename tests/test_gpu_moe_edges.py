"""GPU checks of the MoE operators and the GEMM epilogues at the edges of their contracts: no tokens,
extreme logits, results in place, values that are not finite."""
import numpy as np
import pytest
import torch

import oracle
import synth
import moe_grouped_gemm_02_gb300 as dg
from oracle import moe
from tests._parity import assert_within_tolerance, bits, to_dev

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "silu", "swiglu"]


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------------------------
# A rank that got no tokens
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
def test_epilogues_without_rows(act):
    N, K, G, H = 272, 256, 3, 136 if act == "swiglu" else 272
    u8, i32 = torch.uint8, torch.int32
    kp, al = dg.packed_sf_shape(None, N, K)
    b, sfb = torch.zeros((G, N, K), dtype=u8, device="cuda"), torch.zeros((G, kp, al), dtype=i32, device="cuda")
    a, sfa, bias = _empty(0, K, dtype=u8), _empty(kp, 0, dtype=i32), torch.zeros((G, N), device="cuda")
    d, z = _empty(0, H), _empty(0, N)
    assert a.data_ptr() == 0                                    # torch's empty tensors have a null pointer
    dg.dg_fp8_gemm_nt_act(a, sfa, b[0], sfb[0], d, act=act, bias=bias[0], residual=d, z=z)
    dg.dg_m_grouped_fp8_gemm_nt_contiguous_act(a, sfa, b, sfb, d, _empty(0, dtype=i32), act=act, bias=bias, residual=d, z=z)
    n = torch.zeros((G,), dtype=i32, device="cuda")
    dg.dg_m_grouped_fp8_gemm_nt_masked_act(_empty(G, 0, K, dtype=u8), _empty(G, kp, 0, dtype=i32), b, sfb, _empty(G, 0, H), n,
                                          act=act, bias=bias, residual=_empty(G, 0, H), z=_empty(G, 0, N))
    db = torch.full((G, N), 7.0, device="cuda")
    dg.dg_act_backward(d, z, _empty(0, N), act=act, dbias=db, workspace=_empty(0, N, dtype=torch.float32),
                       m_indices=_empty(0, dtype=i32))
    dg.dg_check_device_error()
    assert torch.all(db == 0)


def test_layer_without_tokens():
    # forward and backward of the example layer on a rank without tokens: every weight's gradient is zeros
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.MoELayer(hidden=256, ffn=128, experts=3, choices=2)
    x = _empty(0, 256)
    y, kept = layer.forward(x)
    grads = layer.backward(torch.empty_like(x), kept)
    dg.dg_check_device_error()
    assert y.shape == (0, 256) and grads.pop("x").shape == (0, 256)
    assert set(grads) == {"router", "w1", "w2", "b1", "b2"} and all(torch.all(g == 0) for g in grads.values())
