"""8-bit integer rows and the gated sandwich norm without a GPU: the oracle's own pins
and the refusals of the C entry points (all made on the host, before any CUDA call)."""

import ctypes

import numpy as np
import pytest

from oracle import int8 as I8
from oracle import layers as OL
from oracle import plan as OP
from shared_token_transformer_b200 import binding as B
from shared_token_transformer_b200 import build as Bd

P = 1 << 20          # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def built():
    Bd.build()


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def test_rows_are_reproduced_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(rng.uniform(-30, 30, (50, 1)))
    x = x.astype(np.float32).astype(np.float64)
    q, s = I8.quantize_rows(x)
    assert np.abs(q).max() == 127 and np.all(q == np.rint(q))
    # half a step, and the fp32 rounding of inv (2^-24) over up to 127 steps
    assert np.all(np.abs(q * s[:, None] - x) <= s[:, None] * (0.5 + 2 * 127 * 2.0 ** -24))


def test_special_rows():
    x = np.zeros((5, 8))
    x[1] = 2.0 ** -120
    x[2, 3] = np.inf
    x[3, 0] = np.nan
    x[4] = [254, 127, 1, 3, -3, -1, 0, 5]      # scale 2: ties at odd values go to the even integer
    q, s = I8.quantize_rows(x)
    assert s[0] == s[1] == 1 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 2
    assert not q[:4].any()
    np.testing.assert_array_equal(q[4], [127, 64, 0, 2, -2, 0, 0, 2])


def test_sandwich_without_norms_gates_and_scales_is_the_layer():
    rng = np.random.default_rng(1)
    plan = OP.make_plan((1, 5, 6), (1, 4, 4), (1, 2, 2))
    m = OL.Model(16, 1, 32, (0, 8, 8))
    p = {"w_qkv": rng.standard_normal((48, 16)), "w_o": rng.standard_normal((16, 16)),
         "w_1": rng.standard_normal((32, 16)), "w_2": rng.standard_normal((16, 32)),
         "b_qkv": rng.standard_normal(48), "b_o": rng.standard_normal(16), "b_1": rng.standard_normal(32),
         "b_2": rng.standard_normal(16), "ln1_g": rng.standard_normal(16), "ln1_b": rng.standard_normal(16),
         "ln2_g": rng.standard_normal(16), "ln2_b": rng.standard_normal(16), "q_g": np.ones(16), "k_g": np.ones(16)}
    S = rng.standard_normal((plan.U + plan.T, 16))
    np.testing.assert_allclose(OL.block_shared_sandwich(S, p, {}, m, plan), OL.block_shared(S, p, m, plan), rtol=1e-12)
    X = OL.gather(S, plan)
    np.testing.assert_allclose(OL.block_tiled_sandwich(X, p, {}, m, plan), OL.block_tiled(X, p, m, plan), rtol=1e-12)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
INT8 = lambda block="ln_gelu": B.model_desc(256, 4, 256, "int8", (0, 32, 32), block=block)   # noqa: E731


def q8_args(**kw):
    a = dict(model=INT8(), x=P, xs=P, rows=4, K=64, W=P, ws=P, N=64, bias=P, epi=0, y=P)
    a.update(kw)
    return a


def call_q8(a):
    return B.lib().ts_op_linear_q8(ctypes.byref(a["model"]), a["x"], a["xs"], a["rows"], a["K"], a["W"], a["ws"], a["N"],
                                   a["bias"], a["epi"], a["y"], None)


@pytest.mark.parametrize("bad,status", [
    ({"x": None}, 1), ({"xs": None}, 1), ({"W": None}, 1), ({"ws": None}, 1), ({"bias": None}, 1), ({"y": None}, 1),
    ({"x": P + 8}, 1), ({"xs": P + 4}, 1), ({"W": P + 1}, 1), ({"y": P + 2}, 1), ({"ws": P + 4}, 1),
    ({"rows": -1}, 1), ({"K": 0}, 1), ({"N": 0}, 1), ({"epi": 4}, 1), ({"epi": -1}, 1),
    ({"K": 72}, 2), ({"K": 24}, 2), ({"N": 4}, 2), ({"N": 100}, 2), ({"K": 131072}, 2),
    ({"model": B.model_desc(256, 4, 256, "bf16", (0, 32, 32))}, 1),
    ({"model": B.model_desc(64, 4, 256, "f32", (0, 8, 8))}, 1),
    ({"model": B.model_desc(256, 4, 256, "fp8", (0, 32, 32))}, 2),      # e4m3 needs K % 128 == 0
    ({"model": B.model_desc(250, 5, 256, "int8", (0, 32, 18))}, 2),
])
def test_linear_q8_refuses(bad, status):
    assert call_q8(q8_args(**bad)) == status
    assert B.lib().ts_last_error()


@pytest.mark.parametrize("bad,status", [
    ({"K": 72}, 2), ({"N": 12}, 2), ({"K": 131072}, 2), ({"scratch": None}, 1), ({"scratch": P + 8}, 1), ({"ws": None}, 1),
    ({"ws": P + 4}, 1),
])
def test_int8_linear_refuses(bad, status):
    a = q8_args(scratch=P)
    a.update(bad)
    st = B.lib().ts_op_linear(ctypes.byref(a["model"]), a["x"], a["rows"], a["K"], a["W"], a["ws"], a["N"], a["bias"],
                              a["epi"], a["y"], a["scratch"], None)
    assert st == status


def test_e4m3_and_bf16_linear_refuse_sizes_before_anything_runs():
    for dt, K in (("fp8", 100), ("bf16", 100), ("fp8", 64)):
        m = B.model_desc(256, 4, 256, dt, (0, 32, 32))
        assert B.lib().ts_op_linear(ctypes.byref(m), P, 4, K, P, P, 64, P, 0, P, P, None) == 2


def test_no_rows_is_no_work():
    assert call_q8(q8_args(rows=0)) == 0
    assert B.lib().ts_quantize_rows_i8(P, 0, 8, P, P, None) == 0
    ng = B.NormGate()
    assert B.lib().ts_op_norm_gate(ctypes.byref(INT8()), ctypes.byref(ng), P, P, None, 0, P, None, None, None) == 0


@pytest.mark.parametrize("x,rows,cols,q,s", [(None, 1, 8, P, P), (P, 1, 8, None, P), (P, 1, 8, P, None),
                                             (P, -1, 8, P, P), (P, 1, 0, P, P), (P, 1, 12, P, P), (P + 8, 1, 8, P, P),
                                             (P, 1, 8, P + 8, P), (P, 1, 8, P, P + 4)])
def test_quantize_refuses(x, rows, cols, q, s):
    assert B.lib().ts_quantize_rows_i8(x, rows, cols, q, s, None) == 1


def call_ng(model=None, x=P, y=P, group=None, rows=2, x_out=P, xn=P, xs=None, null=False, **vec):
    ng = B.NormGate()
    for k, v in dict({"post_g": P, "post_b": P, "pre_g": P, "pre_b": P, "gate": P, "scale": P, "groups": 1}, **vec).items():
        setattr(ng, k, v)
    model = INT8() if model is None else model
    return B.lib().ts_op_norm_gate(ctypes.byref(model), None if null else ctypes.byref(ng), x, y, group, rows, x_out, xn,
                                   xs, None)


@pytest.mark.parametrize("bad", [
    {"null": True}, {"x": None}, {"y": None}, {"x_out": None}, {"rows": -1}, {"x": P + 8}, {"y": P + 2}, {"x_out": P + 4},
    {"xn": P + 8}, {"xs": P + 4}, {"group": P + 2}, {"xn": None}, {"pre_g": None, "pre_b": None}, {"post_b": None},
    {"pre_b": None}, {"post_g": P + 4}, {"gate": P + 8}, {"scale": P + 4}, {"pre_b": P + 4}, {"groups": 0},
    {"groups": -3}, {"xn": None, "pre_g": None, "xs": P},
    {"model": B.model_desc(256, 4, 256, "bf16", (0, 32, 32)), "xs": P},
    {"model": B.model_desc(64, 4, 256, "f32", (0, 8, 8)), "xs": P},
])
def test_norm_gate_refuses(bad):
    assert call_ng(**bad) == 1


def test_sandwich_blocks_refuse_before_anything_runs():
    p = B.Plan((1, 14, 14), (1, 8, 8), (1, 6, 6), host_only=True)
    m, w, sw = B.model_desc(64, 4, 256, "f32", (0, 8, 8)), B.LayerWeights(), B.SandwichWeights()
    for fn in (B.lib().ts_block_shared_sandwich, B.lib().ts_block_tiled_sandwich):
        assert fn(p.handle, ctypes.byref(m), ctypes.byref(w), ctypes.byref(sw), P, P, 1 << 30, None) in (1, 4)
        assert fn(None, ctypes.byref(m), ctypes.byref(w), ctypes.byref(sw), P, P, 1 << 30, None) == 1
    p.close()


def test_int8_model_has_the_e4m3_workspace():
    p = B.Plan((1, 48, 48), (1, 16, 16), (1, 12, 12), host_only=True)
    size = {dt: B.workspace_size(p, B.model_desc(512, 8, 2048, dt, (0, 32, 32)), 8, 2) for dt in ("bf16", "fp8", "int8")}
    assert size["int8"] == size["fp8"] > size["bf16"]
    p.close()


def test_gates_of_different_groups_are_refused():
    import torch
    with pytest.raises(ValueError):
        B.sandwich_weights(gate1=torch.zeros(2, 64), gate2=torch.zeros(3, 64))
    with pytest.raises(ValueError):
        B.norm_gate_desc(post_g=torch.zeros(64), scale=torch.zeros(32))
    with pytest.raises(ValueError):
        B.norm_gate_desc(post_g=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.norm_gate_desc(gate=torch.zeros(64, 2).t())
    g = B.norm_gate_desc(gate=torch.zeros(2, 64), scale=torch.zeros(64))
    assert (g.groups, g.width) == (2, 64)
