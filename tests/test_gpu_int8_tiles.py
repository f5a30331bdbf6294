"""The integer GEMM at every tile width with every epilogue: sizes at which each CTA (or pair of them) walks several
tiles, ragged in rows and columns, and the QKV epilogue elementwise against the 64-bit formula.

The width is normally picked by a cost rule, so a width's tests would silently move to another kernel if the costs
changed.  Child processes therefore force it (TS_GEMM_BN), and the parent runs sizes that the rule decides."""

import dataclasses
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from _gpu import dev, host
from oracle import int8 as I8
from oracle import layers as OL
from oracle import plan as OP
from shared_token_transformer_b200 import binding as B
from shared_token_transformer_b200 import workloads as W
from test_gpu_int8_norm_gate import BF, EPIS, F32, check_linear, i8, layer_on_device, linear_reference, model

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device_status_is_clean():
    yield
    torch.cuda.synchronize()
    B.device_status()


# ---------------------------------------------------------------------------
# few-row kernel: three chunks of K a warp, at 9-16 and 17-32 rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,K,N", [(12, 6144, 1536), (16, 8192, 520), (29, 6160, 264), (32, 4112, 72)])
@pytest.mark.parametrize("epi", ["bias", "gelu", "resid", "swiglu"])
def test_few_rows_of_a_long_k(M, K, N, epi):
    check_linear(M, K, N, epi, seed=M + K + N)


# ---------------------------------------------------------------------------
# large products, by sampled rows
# ---------------------------------------------------------------------------
def tile_rows(M, rng):
    """The first and the last row of every 128-row tile, and forty others."""
    return np.unique(np.concatenate([np.arange(0, M, 128), np.arange(127, M, 128), [M - 1], rng.integers(0, M, 40)]))


@pytest.mark.parametrize("M,K,N", [(16409, 1040, 4080), (14086, 6144, 1536)])
@pytest.mark.parametrize("epi", ["bias", "gelu", "resid", "swiglu"])
def test_large_products(M, K, N, epi):
    """Sizes of the 2K image and of the video with a remainder on every side: tiles of 256 x 256 by pairs of SMs."""
    if epi == "swiglu":
        N //= 2
    rng = np.random.default_rng(M + N)
    wide = 2 * N if epi == "swiglu" else N
    x, wq = rng.integers(-128, 128, (M, K), dtype=np.int8), rng.integers(-127, 128, (wide, K), dtype=np.int8)
    sx = (rng.uniform(0.5, 2, M) / 127).astype(np.float32)
    sw = (0.06 * rng.uniform(0.5, 2, wide) / 127).astype(np.float32)
    b = W.round_to(0.1 * rng.standard_normal(wide), "f32")
    y0 = dev(rng.standard_normal((M, N)), torch.bfloat16)
    y = torch.full((M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    y[:M] = y0
    B.op_linear_q8(model("rms_swiglu" if epi == "swiglu" else "ln_gelu"), i8(x), dev(sx, torch.float32), i8(wq),
                   dev(sw, torch.float32), dev(b, torch.float32), y[:M], EPIS[epi])
    rows = tile_rows(M, rng)
    want, tol = linear_reference(x[rows], sx[rows].astype(np.float64), wq, sw.astype(np.float64), b, epi, host(y0[rows]))
    ok = np.abs(host(y[rows]) - want) <= tol
    assert ok.all(), (rows[np.argwhere(~ok)[:5, 0]], np.argwhere(~ok)[:5, 1])
    assert (y[M:] == 9.0).all()


# ---------------------------------------------------------------------------
# the QKV epilogue
# ---------------------------------------------------------------------------
def turned(v, e, pos, m):
    """RoPE of values v and of their error bounds e [n, heads, hd]: |cos| and |sin| at most carry the pair's errors over,
    cos and sin are off by 2^-24 of one each and the two products and the sum by 2^-24 each."""
    at = OL.rope(v, pos, m)
    out = np.empty_like(e)
    off = 0
    for D in m.rope_dims:
        a, b = slice(off, off + D // 2), slice(off + D // 2, off + D)
        size = np.abs(v[:, :, a]) + np.abs(v[:, :, b])
        both = np.hypot(e[:, :, a], e[:, :, b])      # max of |cos| ea + |sin| eb
        out[:, :, a] = out[:, :, b] = both + 4 * F32 * size
        off += D
    return at, out


def qkv_reference(x, p, m, pos, turn):
    """(q, k, v) [n, d] of rows x and elementwise bounds.

    The norm is off by dn (a sum of at most 64 terms in a lane and five steps across lanes, as in a seam).  Its row's
    scale follows by dn / 127, and an integer may be the other one where the value lies that close to a border
    between two: each such value moves the sum by its |w|.  Then 2^-24 for each fp32 operation and half a bf16
    step.  Rows with `turn` are rotated by pos."""
    g, b = p["ln1_g"], p["ln1_b"]
    rms = m.block == "rms_swiglu"
    n1 = OL.block_norm(x, g, b, m)
    c = 0.0 if rms else x.mean(1, keepdims=True)
    std = np.sqrt(((x - c) ** 2).mean(1, keepdims=True))
    n = np.abs(x - c) / std
    e = 70 * F32 * (np.abs(x).mean(1, keepdims=True) / std + n) + 6 * F32 * (n + np.abs(x) / std)
    dn = np.abs(g) * e + 2 * F32 * (np.abs(g) * n + (0.0 if rms else np.abs(b)))
    top = np.abs(n1).max(1, keepdims=True)
    dtop = dn.max(1, keepdims=True)
    q, s = I8.quantize_rows(n1)
    t = n1 * (127.0 / top)
    dt = dn * 127.0 / top + np.abs(t) * (dtop / top + 3 * F32)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= dt
    wq, sw = I8.quantize_rows(p["w_qkv"])
    acc = (q @ wq.T) * s[:, None] * sw
    z = acc + p["b_qkv"]
    dz = (near @ np.abs(wq).T) * s[:, None] * sw + np.abs(acc) * (dtop / top + 2 * F32) + 4 * F32 * (np.abs(acc) + np.abs(p["b_qkv"]))
    dz *= 1.001                                       # products of two errors
    out = []
    for i, gain in enumerate((p["q_g"], p["k_g"], None)):
        v, dv = (a[:, i * m.d:(i + 1) * m.d].reshape(len(x), m.heads, m.hd) for a in (z, dz))
        if gain is not None:
            r = np.sqrt((v * v).mean(-1, keepdims=True) + m.eps_qk)
            dr = np.sqrt((dv * dv).mean(-1, keepdims=True))          # the norm of the error bounds the norm's error
            w = OL.rms_norm(v, gain, m.eps_qk)
            dw = np.abs(gain) / r * dv + np.abs(w) * dr / r * 1.01 + 70 * F32 * np.abs(w)
            at, dat = turned(w, dw, pos, m)
            v, dv = np.where(turn[:, None, None], at, w), np.where(turn[:, None, None], dat, dw)
        out.append((v.reshape(len(x), -1), (dv + BF * (np.abs(v) + dv)).reshape(len(x), -1)))
    return out


def check_qkv(cfg, mode):
    op = OP.make_plan(cfg.grid, cfg.win, cfg.stride, registers=cfg.R)
    plan = B.Plan(cfg.grid, cfg.win, cfg.stride, registers=cfg.R)
    dr = W.Draw(cfg, op.T, seed=3, affine=True)
    S = np.concatenate(dr.states())
    p = dr.layer()
    om = OL.Model(cfg.d, cfg.heads, cfg.mlp, cfg.rope_dims, int8=True, block=cfg.block)
    m = B.model_desc(cfg.d, cfg.heads, cfg.mlp, "int8", cfg.rope_dims, block=cfg.block)
    w = B.layer_weights(layer_on_device(cfg, p))
    if mode == B.TS_ROWS_SHARED:
        state = S
        f, y, x = np.unravel_index(np.arange(op.U), cfg.grid)
        pos = np.concatenate([np.stack([f, y, x], 1), np.repeat(plan.origins, op.R, axis=0)])
        turn = np.ones(len(S), bool)
    else:
        state = OL.gather(S, op).reshape(-1, cfg.d)
        one = np.concatenate([np.zeros((op.R, 3), np.int64), op.slot_pos])
        pos = np.tile(one, (op.T, 1))
        turn = np.tile(np.arange(op.N) >= op.R, op.T)
    n, d = state.shape
    out = torch.full((n + 2, 3 * d), 9.0, dtype=torch.bfloat16, device="cuda")
    table = 4 * sum(g * r for g, r in zip(cfg.grid, cfg.rope_dims))
    scratch = torch.empty(3 * n * d + 4 * n + table + 1024, dtype=torch.uint8, device="cuda")
    B.op_qkv(plan, m, w, mode, dev(state, torch.bfloat16), out[:n], scratch)
    rows = tile_rows(n, np.random.default_rng(n))
    got = host(out[rows])
    for i, (want, tol) in enumerate(qkv_reference(state[rows], p, om, pos[rows], turn[rows])):
        part = got[:, i * d:(i + 1) * d]
        ok = np.abs(part - want) <= tol
        assert ok.all(), ("qkv"[i], (~ok).sum(), rows[np.argwhere(~ok)[:5, 0]], part[~ok][:5], want[~ok][:5], tol[~ok][:5])
        assert np.median(tol / np.maximum(np.abs(want), 1e-2)) < 0.05      # the bound tells a wrong value
    assert (out[n:] == 9.0).all()
    plan.close()


def int8(name, **kw):
    return dataclasses.replace(W.CONFIGS[name], name=name + "_int8", dtype="int8", **kw)


@pytest.mark.parametrize("mode", [B.TS_ROWS_SHARED, B.TS_ROWS_TILED])
@pytest.mark.parametrize("cfg", [int8("video44x80_bf16"), int8("image2k_bf16", block="rms_swiglu"), int8("stack48_bf16", R=3)],
                         ids=lambda c: c.name)
def test_qkv_values(cfg, mode):
    check_qkv(cfg, mode)


# ---------------------------------------------------------------------------
# every width, forced
# ---------------------------------------------------------------------------
FORCED = '''
import sys
sys.path[:0] = ["tests", "."]
import dataclasses, torch
import test_gpu_int8_tiles as T
from shared_token_transformer_b200 import binding as B, workloads as W
for epi in T.EPIS:
    for M, K, N in {sizes}:
        T.check_linear(M, K, N // 2 if epi == "swiglu" else N, epi, seed=M + K)
vol = W.small_config("vol", grid=(3, 9, 12), win=(2, 6, 8), stride=(1, 3, 4), d=256, heads=4, mlp=512, dtype="int8",
                     rope_dims=(16, 24, 24))
for cfg in (vol, dataclasses.replace(W.CONFIGS["stack48_bf16"], dtype="int8")):
    for mode in (B.TS_ROWS_SHARED, B.TS_ROWS_TILED):
        T.check_qkv(cfg, mode)
torch.cuda.synchronize()
B.device_status()
print("forced and right")
'''


@pytest.mark.parametrize("bn,sizes", [(256, [(5020, 144, 3008), (300, 1040, 528), (700, 16, 272), (33, 2064, 272)]),
                                      (128, [(5100, 144, 1520), (300, 1040, 528), (700, 16, 272), (33, 2064, 272)]),
                                      (64, [(5100, 144, 752), (300, 1040, 528), (700, 16, 272), (33, 2064, 272)])])
def test_every_width_with_every_epilogue(bn, sizes):
    """The first size gives each CTA, or pair of them, at least three tiles: rings, accumulators, scales and residual boxes
    are used again."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FORCED.format(sizes=sizes)], cwd=root, capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, TS_GEMM_BN=str(bn)))
    assert r.returncode == 0 and "forced and right" in r.stdout, (r.stdout[-500:], r.stderr[-3000:])


FIRST_CAPTURE_OF_PAIRS = '''
import torch
from shared_token_transformer_b200 import binding as B
calls = []
for block, epi, want in (("ln_gelu", 0, 2.0), ("ln_gelu", 1, 1.9545), ("ln_gelu", 2, 5.0), ("rms_swiglu", 3, 3.5232)):
    m = B.model_desc(256, 4, 256, "int8", (0, 32, 32), block=block)
    M, K, N = 700, 256, 512
    wide = 2 * N if epi == 3 else N
    x, w = (torch.ones((n, K), dtype=torch.int8, device="cuda") for n in (M, wide))
    xs, s, b = torch.full((M,), 1.0 / 128, device="cuda"), torch.ones(wide, device="cuda"), torch.zeros(wide, device="cuda")
    y = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    calls.append((m, x, xs, w, s, b, y, epi, want))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for c in calls:
        B.op_linear_q8(*c[:8])
g.replay()
torch.cuda.synchronize()
B.device_status()
for c in calls:
    assert (c[6].double() - c[8]).abs().max().item() <= c[8] * 2.0 ** -7, (c[7], c[6].flatten()[:4])
print("captured first")
'''


def test_first_calls_of_the_pair_kernel_inside_a_capture():
    """z = 256 / 128 = 2: bias 2, GELU 1.9545, residual 3 + 2, SwiGLU silu(2) * 2 = 3.5232."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURE_OF_PAIRS], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, TS_GEMM_BN="256"))
    assert r.returncode == 0 and "captured first" in r.stdout, (r.stdout, r.stderr[-2000:])
