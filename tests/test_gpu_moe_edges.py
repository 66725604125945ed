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


def test_masked_layout_without_tokens():
    # a decode step of no tokens: a layout of no rows per group
    G, K, k = 5, 256, 2
    i32 = torch.int32
    idx, pos, w, n = _empty(0, k, dtype=i32), _empty(0, k, dtype=i32), _empty(0, k, dtype=torch.float32), torch.full((G,), 7, dtype=i32, device="cuda")
    dg.dg_moe_route(_empty(0, G, dtype=torch.float32), idx, w)
    dg.dg_moe_sort_masked(idx, pos, n, 0)
    assert n.tolist() == [0] * G
    x, y = _empty(0, K), _empty(0, K)
    dg.dg_moe_dispatch_fp8(x, pos, _empty(G, 0, K, dtype=torch.uint8), _empty(*dg.packed_sf_shape(G, 0, K), dtype=i32))
    dg.dg_moe_combine(_empty(G, 0, K), pos, w, y, residual=x)
    with pytest.raises(dg.DGError):
        dg.dg_moe_sort_masked(torch.zeros((1, k), dtype=i32, device="cuda"), _empty(1, k, dtype=i32), n, 0)
    with pytest.raises(dg.DGError):
        dg.dg_moe_sort_masked(idx, pos, n, -1)


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


# ---------------------------------------------------------------------------------------------
# Epilogues: the residual in place, values that are not finite
# ---------------------------------------------------------------------------------------------
def _operands(lead_a, lead_b, rows, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    # codes of +-[2^-3, 7.5]: finite, so sums of any order differ in rounding only; scales 2^-4 .. 2^-1
    a, b = (torch.randint(0x20, 0x50, (*s, K), generator=g, device="cuda").to(torch.uint8) |
            (torch.randint(0, 2, (*s, K), generator=g, device="cuda") << 7).to(torch.uint8) for s in ((*lead_a, rows), (*lead_b, N)))
    def scales(lead, r):
        kp, al = dg.packed_sf_shape(None, r, K)
        by = torch.randint(123, 127, (*lead, kp, al, 4), generator=g, device="cuda")
        return (by << torch.tensor([0, 8, 16, 24], device="cuda")).sum(-1).to(torch.int32)
    return a, scales(lead_a, rows), b, scales(lead_b, N)


def _case(layout, rows, G, N, K, act, seed=1):
    """call(d, **extras) of one layout, D's shape and z's."""
    lead = (G,) if layout == "masked" else ()
    a, sfa, b, sfb = _operands(lead, () if layout == "dense" else (G,), rows, N, K, seed)
    H = N // 2 if act == "swiglu" else N
    if layout == "dense":
        return (lambda d, **x: dg.dg_fp8_gemm_nt_act(a, sfa, b, sfb, d, act=act, **x)), (rows, H), (N,)
    if layout == "contiguous":
        # expert e: 128 rows for every second block, the last of them padded
        m = torch.arange(rows, device="cuda").div(256, rounding_mode="floor").clamp(max=G - 1).to(torch.int32)
        m[rows - 37:] = -1
        return (lambda d, **x: dg.dg_m_grouped_fp8_gemm_nt_contiguous_act(a, sfa, b, sfb, d, m, act=act, **x)), (rows, H), (G, N)
    m = torch.tensor([rows, 1, 0, rows - 3][:G], dtype=torch.int32, device="cuda")
    return (lambda d, **x: dg.dg_m_grouped_fp8_gemm_nt_masked_act(a, sfa, b, sfb, d, m, act=act, **x)), (G, rows, H), (G, N)


# layout, rows, G, N, K, configuration, split, SMs (0: all): every way the epilogues read the residual, with one tile per CTA and with several
PLANS = [("dense", 300, 1, 720, 384, c, 1, s) for c in ("config_bn224_s3_m2", "config_bn192_s3_m2", "config_bn192_s5_k2", "config_bn128_s5_k2",
                                                        "config_bn224_s4_a2", "config_bn64_s8_a2", "config_bn32_s8_a2") for s in (0, 4)] + \
        [("dense", 61, 1, 720, 384, "config_bn128_s8_k2_r64", 1, s) for s in (0, 4)] + \
        [("dense", 130, 1, 464, 2048, c, p, s) for c in ("config_bn128_s5_k2", "config_bn64_s8_a2", "config_bn32_s8_a2")
         for p, s in ((2, 0), (4, 16), (8, 0))] + \
        [("dense", 50, 1, 464, 2048, "config_bn128_s8_k2_r64", p, s) for p, s in ((2, 16), (8, 0))] + \
        [("contiguous", 896, 4, 464, 640, c, 1, s) for c in ("config_bn224_s3_m2", "config_bn192_s3_m2", "config_bn128_s5_k2", "config_bn224_s4_a2")
         for s in (0, 4)] + \
        [("masked", 200, 4, 320, 1024, c, p, s) for c, p, s in (("config_bn128_s5_k2", 1, 0), ("config_bn128_s5_k2", 4, 0),
                                                                 ("config_bn224_s4_a2", 1, 4), ("config_bn64_s8_a2", 2, 16))] + \
        [("masked", 600, 2, 320, 512, "config_bn224_s3_m2", 1, s) for s in (0, 4)]


def _planned(monkeypatch, cfg, split, sms):
    monkeypatch.setenv("DG_FORCE_CONFIG", cfg)
    monkeypatch.setenv("DG_FORCE_SPLIT", str(split))
    dg.dg_set_num_sms(sms)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout,rows,G,N,K,cfg,split,sms", PLANS)
def test_residual_in_place(act, layout, rows, G, N, K, cfg, split, sms, monkeypatch):
    # D as its own residual: the bits of the call with a residual of its own
    call, shape, bias_shape = _case(layout, rows, G, N, K, act)
    g = torch.Generator(device="cuda").manual_seed(2)
    res = (3 * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)
    bias = torch.randn(bias_shape, generator=g, device="cuda")
    apart, inplace = res.clone(), res.clone()           # (rows that the call leaves alone are the same in both)
    _planned(monkeypatch, cfg, split, sms)
    try:
        call(apart, bias=bias, residual=res)
        call(inplace, bias=bias, residual=inplace)
    finally:
        dg.dg_set_num_sms(0)
    dg.dg_check_device_error()
    assert torch.equal(apart.view(torch.int16), inplace.view(torch.int16))
    assert not torch.equal(apart, res)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout,rows,G,N,K,cfg,split,sms", PLANS)
def test_values_that_are_not_finite_stay_in_their_place(act, layout, rows, G, N, K, cfg, split, sms, monkeypatch):
    # a bias of infinities and NaN in one column of some pairs (the first or the second): the other columns
    # hold the same values as without, and the column itself the activation's limit.  SiLU and GELU divide by the
    # product of a pair's denominators, so the column beside it may round to the next BF16 value; all others hold
    # the same bits
    call, shape, bias_shape = _case(layout, rows, G, N, K, act)
    bias = torch.randn(bias_shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    odd = bias.clone()
    cols = torch.arange(0, N, 6, device="cuda") + (torch.arange(0, N, 6, device="cuda") // 6) % 2
    cols = cols[cols < N]
    kinds = torch.arange(cols.numel(), device="cuda") // 2 % 3
    values = torch.tensor([float("inf"), float("-inf"), float("nan")], device="cuda")
    odd[..., cols] = values[kinds]
    d0, d1 = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    _planned(monkeypatch, cfg, split, sms)
    try:
        call(d0, bias=bias)
        call(d1, bias=odd)
    finally:
        dg.dg_set_num_sms(0)
    dg.dg_check_device_error()
    at = cols // 2 if act == "swiglu" else cols
    clean = torch.ones((shape[-1],), dtype=torch.bool, device="cuda")
    clean[at] = False
    apart = (d0[..., clean].view(torch.int16).int() - d1[..., clean].view(torch.int16).int()).abs()
    assert int(apart.max()) <= (1 if act in ("silu", "gelu") else 0)
    beside = torch.zeros_like(clean)
    beside[at ^ 1] = True
    assert int(apart[..., ~beside[clean]].max()) == 0
    assert bool(d0.isfinite().all())
    if act == "swiglu":
        return
    live = d0.abs().sum(-1) > 0                         # rows that the call computes
    got = d1[live][:, cols].float()
    assert bool(live.any())
    low = {"none": float("-inf"), "relu": 0.0}.get(act)
    assert bool((got[:, kinds == 0] == float("inf")).all()) and bool(got[:, kinds == 2].isnan().all())
    assert bool((got[:, kinds == 1] == low).all() if low is not None else (got[:, kinds == 1].abs() <= 1e-17).all())
