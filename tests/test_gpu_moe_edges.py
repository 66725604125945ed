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


# ---------------------------------------------------------------------------------------------
# Router: extreme logits
# ---------------------------------------------------------------------------------------------
EPS = 2.0 ** -24


def _sigmoid(x):
    # in 64 bits, to a few of their units at either end
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def _as(x, dtype):
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.cuda(), t.double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_slope_of_large_logits(dtype, renorm):
    # dl_c = scale q_c (1 - s_c) (dw_c - mean): the slope 1 - s is e^-x for a large logit x.  A score or a slope
    # is an exponential (2 units), a sum, a quotient and a product; q one quotient and two sums over k more: below
    # 64 eps of q (1 - s) (|dw| + sum |dw q|), BF16 logits' gradients rounded once more
    T, E, k = 48, 16, 8
    r = _rng(31)
    x = r.uniform(8, 30, (T, E)) * np.where(r.random((T, E)) < 0.25, -1, 1)
    x[:, 0] = r.uniform(-2, 2, T)
    x, xv = _as(x, dtype)
    idx, w = _empty(T, k, dtype=torch.int32), _empty(T, k, dtype=torch.float32)
    dg.dg_moe_route(x, idx, w, scoring="sigmoid", renormalize=renorm, scale=2.5)
    dw = r.standard_normal((T, k)).astype(np.float32)
    dl = torch.full((T, E), 7.0, dtype=x.dtype, device="cuda")
    dg.dg_moe_route_backward(x, idx, to_dev(dw), dl, scoring="sigmoid", renormalize=renorm, scale=2.5)
    at = idx.long().cpu().numpy()
    chosen = np.take_along_axis(xv, at, 1)
    s, slope, g = _sigmoid(chosen), _sigmoid(-chosen), dw.astype(np.float64)
    q = s / s.sum(1, keepdims=True) if renorm else s
    mean = (g * q).sum(1, keepdims=True) if renorm else 0.0
    size = np.abs(g) + (np.abs(g * q).sum(1, keepdims=True) if renorm else 0.0)
    want, bound = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, at, 2.5 * q * slope * (g - mean), 1)
    np.put_along_axis(bound, at, 64 * EPS * 2.5 * q * slope * size, 1)
    if dtype == "bf16":
        bound += 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(dl.double().cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_renormalised_sigmoid_of_scores_that_underflow(dtype):
    # every chosen logit so far below zero that its sigmoid has no FP32 value: the weights are the scores'
    # ratios all the same (down to logits of -700: below, masks, the scores are 0).  Differences of logits are rounded to 2^-22 at most (spread 8: 4 eps of the
    # exponential); with the rest of the arithmetic as above, 64 eps
    k, E = 6, 16
    r = _rng(41)
    centre = np.repeat([-87.5, -88.5, -95.0, -104.0, -200.0, -1e4, -3e38], 5)[:, None]
    x = centre + r.uniform(-8, 0, (35, E))
    x = np.concatenate([x, np.where(np.arange(E) == 3, 3.0, -95.0)[None] + r.uniform(-1, 0, (1, E))])   # one large, the rest far below
    x, xv = _as(x, dtype)
    T = xv.shape[0]
    idx, w = _empty(T, k, dtype=torch.int32), _empty(T, k, dtype=torch.float32)
    dg.dg_moe_route(x, idx, w, scoring="sigmoid", renormalize=True, scale=2.5)
    at = np.argsort(-xv, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), at)
    chosen = np.take_along_axis(xv, at, 1)
    top = np.minimum(chosen[:, :1], 0)
    s = np.where(chosen >= 0, 1.0, np.exp(np.minimum(chosen - top, 0))) / (1 + np.exp(-np.abs(chosen)))
    s[chosen < -700] = 0
    q = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    tiny = 2.0 ** -145                           # (the last row's small scores are subnormal)
    assert np.all(np.abs(w.double().cpu().numpy() - 2.5 * q) <= 64 * EPS * 2.5 * q + tiny)
    dw = r.standard_normal((T, k)).astype(np.float32)
    dl = torch.full((T, E), 7.0, dtype=x.dtype, device="cuda")
    dg.dg_moe_route_backward(x, idx, to_dev(dw), dl, scoring="sigmoid", renormalize=True, scale=2.5)
    g, slope = dw.astype(np.float64), _sigmoid(-chosen)
    want, bound = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, at, 2.5 * q * slope * (g - (g * q).sum(1, keepdims=True)), 1)
    np.put_along_axis(bound, at, 64 * EPS * 2.5 * q * slope * (np.abs(g) + np.abs(g * q).sum(1, keepdims=True)), 1)
    if dtype == "bf16":
        bound += 2.0 ** -8 * np.abs(want) + 2.0 ** -134      # BF16's subnormals are 2^-133 apart
    assert np.all(np.abs(dl.double().cpu().numpy() - want) <= bound + 4 * tiny)


def test_weights_of_equal_logits_are_rounded_once():
    # equal logits: every exponential is exactly 1 and their sum an integer, so the weight is 1 / n, rounded to
    # the nearest FP32 value by the one division
    for E in list(range(1, 400)) + [512, 513, 777, 1000, 1021, 1024]:
        for dtype in (torch.float32, torch.bfloat16):
            x = torch.full((2, E), 0.75, dtype=dtype, device="cuda")
            for k, scoring, renorm, n in ((1, "softmax", False, E), (min(E, 31), "softmax", True, min(E, 31)),
                                          (min(E, 27), "sigmoid", True, min(E, 27))):
                if scoring == "sigmoid":
                    x.zero_()                                          # scores of exactly 1/2
                idx, w = _empty(2, k, dtype=torch.int32), _empty(2, k, dtype=torch.float32)
                dg.dg_moe_route(x, idx, w, scoring=scoring, renormalize=renorm)
                assert np.all(w.cpu().numpy() == np.float32(1) / np.float32(n)), (E, dtype, scoring, renorm)


# ---------------------------------------------------------------------------------------------
# Tensors of another device
# ---------------------------------------------------------------------------------------------
def test_tensors_of_another_device_are_refused():
    # (tensors with a null pointer stand for those of a second GPU: nothing could be launched on them)
    class Far(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} of a tensor without memory")

    def far_tensor(shape, dtype):
        return torch.Tensor._make_wrapper_subclass(Far, shape, dtype=dtype, device=torch.device("cuda", 1))

    far, far_logits, far_w = far_tensor((4, 2), torch.int32), far_tensor((4, 8), torch.float32), far_tensor((4, 2), torch.float32)
    assert far.device.index == 1 and torch.cuda.current_device() == 0
    here = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    n = torch.zeros((4,), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="current CUDA device"):
        dg.dg_moe_sort_masked(far, here, n, 8)
    with pytest.raises(ValueError, match="current CUDA device"):
        dg.dg_moe_sort_masked(here, far, n, 8)
    with pytest.raises(ValueError, match="current CUDA device"):
        dg.dg_moe_route(far_logits, far, far_w)


# ---------------------------------------------------------------------------------------------
# First calls of a process
# ---------------------------------------------------------------------------------------------
FIRST_CALLS = """
import os
import torch
import moe_grouped_gemm_02_gb300 as dg
M, N, K = 256, 512, 512
a, b = (torch.randint(0, 0x70, (r, K), dtype=torch.uint8, device="cuda") for r in (M, N))
sfa, sfb = (torch.full(dg.packed_sf_shape(None, r, K), 0x77777777, dtype=torch.int32, device="cuda") for r in (M, N))
d, d1, d2 = (torch.zeros((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3))
torch.cuda.synchronize()
free = torch.cuda.mem_get_info()[0]
dg.dg_fp8_gemm_nt(a, sfa, b, sfb, d)
torch.cuda.synchronize()
print("plain", free - torch.cuda.mem_get_info()[0])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dg.dg_fp8_gemm_nt_act(a, sfa, b, sfb, d1, act="gelu")
    os.environ["DG_FORCE_CONFIG"] = "config_bn32_s8_a2"
    dg.dg_fp8_gemm_nt_act(a, sfa, b, sfb, d2, act="gelu")
    del os.environ["DG_FORCE_CONFIG"]
g.replay()
dg.dg_fp8_gemm_nt_act(a, sfa, b, sfb, d, act="gelu")
dg.dg_check_device_error()
assert torch.equal(d, d1) and torch.allclose(d.float(), d2.float(), rtol=2.0 ** -7)
print("captured")
"""


def test_plain_gemm_loads_no_epilogue_kernels():
    # a process that only multiplies holds the plain kernels, 4 MB of the device's memory; with the epilogues' it was
    # 16 MB.  And the epilogues' first call may be under capture
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = r.stdout.split()
    assert out[0] == "plain" and out[2] == "captured"
    assert int(out[1]) <= 8 << 20


# ---------------------------------------------------------------------------------------------
# Activation gradient: rows of no expert
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("act", ACTS)
def test_rows_past_the_last_expert_have_no_gradient(act):
    # the GEMM writes zeros to rows whose expert index is outside [0, G), and the bias gradient leaves them out:
    # their dz is zeros too, and neither their z nor their dd is read
    N, G, H = 272, 2, 136 if act == "swiglu" else 272
    m = torch.tensor([0] * 100 + [-1] * 28 + [1] * 128 + [2] * 128 + [4096] * 128, dtype=torch.int32, device="cuda")
    rows = m.numel()
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn((rows, N), generator=g, device="cuda").to(torch.bfloat16)
    dd = torch.randn((rows, H), generator=g, device="cuda").to(torch.bfloat16)
    inside = (m >= 0) & (m < G)
    z[~inside], dd[~inside] = float("nan"), float("nan")
    dz, db = torch.full_like(z, 7.0), torch.full((G, N), 7.0, device="cuda")
    ws = _empty(*dg.act_backward_workspace_shape(rows, N), dtype=torch.float32)
    dg.dg_act_backward(dd, z, dz, act=act, dbias=db, workspace=ws, m_indices=m)
    assert torch.all(dz[~inside] == 0)
    # the inside: bit for bit what the same rows give under -1 padding
    dz2, db2 = torch.empty_like(z), torch.empty_like(db)
    dg.dg_act_backward(dd, z, dz2, act=act, dbias=db2, workspace=ws, m_indices=torch.where(inside, m, -1))
    assert torch.equal(dz[inside], dz2[inside]) and torch.equal(db, db2) and bool(dz[inside].isfinite().all())
