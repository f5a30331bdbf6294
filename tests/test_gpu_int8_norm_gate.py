"""The 8-bit integer linear layer and the gated sandwich norm on the GPU, each against
its formula in 64 bits with elementwise bounds counted from its roundings: half a bf16
step (2^-8 relative) for the output, 2^-24 for each fp32 operation before it."""

import dataclasses

import numpy as np
import pytest
import torch

from _gpu import BIG, SCALE, assert_rows, dev, host, rel_l2
from oracle import int8 as I8
from oracle import layers as OL
from oracle import plan as OP
from shared_token_transformer_b200 import binding as B
from shared_token_transformer_b200 import workloads as W

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -24
EPIS = {"bias": B.TS_EPI_BIAS, "gelu": B.TS_EPI_BIAS_GELU, "resid": B.TS_EPI_BIAS_RESID, "swiglu": B.TS_EPI_BIAS_SWIGLU}


def model(block="ln_gelu", d=256, dtype="int8"):
    return B.model_desc(d, d // 64, 256, dtype, (0, 32, 32), block=block)


def i8(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int8)).cuda()


@pytest.fixture(autouse=True)
def device_status_is_clean():
    yield
    torch.cuda.synchronize()
    B.device_status()


# ---------------------------------------------------------------------------
# rows as 8-bit integers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 16), (7, 264), (333, 1040), (64, 1536), (5, 4096), (9, 6144),
                                       (2, 20000), (2500, 512)])
def test_quantize_rows_exactly(rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1)))
    x[0, : cols // 2] = np.rint(x[0, : cols // 2])
    x = W.round_to(x, "bf16")
    x[-1, 0] = 2 * np.abs(x[-1]).max()             # half the largest magnitude sits on a border (63.5 steps)
    q = torch.full((rows + 1, cols), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), -5.0, device="cuda")
    B.quantize_rows_i8(dev(x, torch.bfloat16), q, s)
    want_q, want_s = I8.quantize_rows(x)
    np.testing.assert_array_equal(host(q)[:rows], want_q)
    np.testing.assert_array_equal(host(s)[:rows], want_s)
    assert (host(q)[rows] == 77).all() and host(s)[rows] == -5.0      # nothing behind the last row


def test_quantize_special_rows():
    x = np.zeros((7, 48))
    x[1] = 2.0 ** -110
    x[2, 30] = np.inf
    x[3, 47] = np.nan
    x[4, :8] = [254, 127, 1, 3, -3, -1, 0, 5]
    x[5, 3] = 2.0 ** -100
    x[6, 5] = -3.0e38
    xb = torch.from_numpy(x).to("cuda", torch.bfloat16)
    q = torch.empty((7, 48), dtype=torch.int8, device="cuda")
    s = torch.empty(7, device="cuda")
    B.quantize_rows_i8(xb, q, s)
    want_q, want_s = I8.quantize_rows(xb.double().cpu().numpy())
    np.testing.assert_array_equal(host(q), want_q)
    np.testing.assert_array_equal(host(s), want_s)


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------
def linear_reference(q, sx, wq, sw, b, epi, y0=None):
    """(value, elementwise bound) of the layer from its integers and scales."""
    acc = (q.astype(np.float64) @ wq.astype(np.float64).T) * sx[:, None] * sw[None, :]
    z = acc + b
    dz = 4 * F32 * (np.abs(acc) + np.abs(b))       # int32 -> fp32, the two scales, the fused add
    if epi == "gelu":
        v = OL.gelu(z)
        dv = 1.13 * dz + 6e-7 * np.maximum(1.0, np.abs(v))       # |gelu'| < 1.13; erf's own error
    elif epi == "swiglu":
        n = z.shape[1] // 2
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        s = OL.silu(g)
        v = s * u
        # |silu'| < 1.1; expf off by (2 + 1.2 |g|) 2^-23 relative, then an add, a division and a product
        dv = np.abs(u) * (1.1 * dg + np.abs(s) * ((2 + 1.2 * np.abs(g)) * 2 + 4) * F32) + np.abs(s) * du
    elif epi == "resid":
        v, dv = z + y0, dz + 2 * F32 * np.abs(z + y0)
    else:
        v, dv = z, dz
    return v, dv + BF * (np.abs(v) + dv) + 1e-38


def check_linear(M, K, N, epi, seed=0, quantised=True, x=None, sx=None, wq=None, sw=None):
    rng = np.random.default_rng(seed)
    wide = 2 * N if epi == "swiglu" else N
    if wq is None:
        wq = rng.integers(-127, 128, (wide, K))
        sw = (0.02 * rng.uniform(0.5, 2, wide) / 127 * 3).astype(np.float32).astype(np.float64)
    b = W.round_to(0.1 * rng.standard_normal(wide), "f32")
    y0 = W.round_to(rng.standard_normal((M, N)), "bf16")
    block = "rms_swiglu" if epi == "swiglu" else "ln_gelu"
    y = torch.full((M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    y[:M] = dev(y0, torch.bfloat16)
    if quantised:
        if x is None:
            x = rng.integers(-128, 128, (M, K))
            sx = (rng.uniform(0.5, 2, M) / 127).astype(np.float32).astype(np.float64)
        q, s = x, sx
        B.op_linear_q8(model(block), i8(x), dev(sx, torch.float32), i8(wq), dev(sw, torch.float32),
                       dev(b, torch.float32), y[:M], EPIS[epi])
    else:
        if x is None:
            x = W.round_to(rng.standard_normal((M, K)), "bf16")
        q, s = I8.quantize_rows(x)
        scratch = torch.full((M * K + 4 * M + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        B.op_linear(model(block), dev(x, torch.bfloat16), i8(wq), dev(b, torch.float32), y[:M], EPIS[epi],
                    w_scale=dev(sw, torch.float32), scratch=scratch)
        assert (scratch[M * K + 4 * M:] == 0x5A).all()      # the documented size is enough
    want, tol = linear_reference(q, s, wq, sw, b, epi, y0)
    got = host(y)
    assert (got[M:] == 9.0).all()                           # nothing behind the last row
    ok = np.abs(got[:M] - want) <= tol
    assert ok.all(), (np.argwhere(~ok)[:5], got[:M][~ok][:5], want[~ok][:5])


SIZES = [(1, 16, 8), (1, 1536, 4608), (2, 64, 64), (6, 6144, 1536), (9, 80, 72), (16, 4096, 1024), (17, 1024, 200),
         (33, 512, 2048), (64, 1536, 520), (65, 1040, 1336), (127, 96, 264), (128, 128, 128), (129, 256, 192),
         (257, 4096, 1024), (333, 1040, 1336), (777, 2048, 512), (2320, 512, 1000), (4099, 272, 776),
         # clusters of two to six CTAs share K: 333, 257, 300, 600 and 64 rows, and a K of fewer slices than CTAs
         (300, 1024, 768), (600, 2048, 264), (40, 6144, 520), (50, 272, 24), (250, 400, 1000),
         # up to 64 rows of a wide W: one CTA a tile
         (33, 2048, 8192), (64, 1040, 5000)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("epi", ["bias", "gelu", "resid", "swiglu"])
def test_linear_q8_int8(M, K, N, epi):
    check_linear(M, K, N, epi, seed=M + K + N)


@pytest.mark.parametrize("M,K,N", [(1, 1536, 4608), (1, 16, 8), (3, 144, 40), (6, 6144, 1536), (20, 512, 264),
                                   (64, 1536, 520), (333, 1040, 1336), (2320, 512, 2048)])
@pytest.mark.parametrize("epi", ["bias", "gelu", "swiglu"])
def test_linear_int8_quantises_rows(M, K, N, epi):
    check_linear(M, K, N, epi, seed=M + K, quantised=False)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_integer_sums_are_exact_at_their_largest(M):
    """K at its limit and every factor -128: the sum 2^14 K needs all 31 bits of int32."""
    K, N = 131056, 16
    x = np.full((M, K), -128)
    wq = np.full((N, K), -128)
    wq[1] = 127
    wq[2, ::2] = 127
    check_linear(M, K, N, "bias", x=x, sx=np.full(M, 2.0 ** -20), wq=wq, sw=np.full(N, 2.0 ** -6))


@pytest.mark.parametrize("M,K", [(9, 256), (20, 256), (200, 1024), (2500, 256)])
@pytest.mark.parametrize("epi", ["bias", "gelu", "swiglu", "resid"])
def test_rows_that_are_not_finite_stay_apart(M, K, epi):
    """A NaN or an infinity in a row makes that row's outputs NaN, through every epilogue and kernel, and no other's."""
    rng = np.random.default_rng(5)
    N = 128
    wide = 2 * N if epi == "swiglu" else N
    x = W.round_to(rng.standard_normal((M, K)), "bf16")
    x[2] = 0.0
    xb = torch.from_numpy(x).to("cuda", torch.bfloat16)
    xb[4, 7] = float("inf")
    xb[6, 0] = float("nan")
    wq = rng.integers(-127, 128, (wide, K))
    sw = np.full(wide, 2.0 ** -10)
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(M * K + 4 * M, dtype=torch.uint8, device="cuda")
    b = W.round_to(rng.standard_normal(wide), "f32")
    B.op_linear(model("rms_swiglu" if epi == "swiglu" else "ln_gelu"), xb, i8(wq), dev(b, torch.float32), y, EPIS[epi],
                w_scale=dev(sw, torch.float32), scratch=scratch)
    got = host(y)
    assert np.isnan(got[[4, 6]]).all()
    rows = [r for r in range(M) if r not in (4, 6)]
    q, s = I8.quantize_rows(x)
    want, tol = linear_reference(q, s, wq, sw, b, epi, np.zeros((M, N)))
    assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all()


def test_linear_q8_e4m3_equals_the_quantising_call():
    rng = np.random.default_rng(8)
    M, K, N = 130, 256, 192
    x, w = (dev(rng.standard_normal(s), torch.bfloat16) for s in ((M, K), (N, K)))
    wq, xq = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K), dtype=torch.uint8, device="cuda")
    sw, sx = torch.empty(N, device="cuda"), torch.empty(M, device="cuda")
    B.quantize_rows_e4m3(w, wq, sw)
    B.quantize_rows_e4m3(x, xq, sx)
    b = dev(rng.standard_normal(N), torch.float32)
    y1, y2 = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.op_linear(model(dtype="fp8"), x, wq, b, y1, w_scale=sw, scratch=torch.empty(M * K + 4 * M, dtype=torch.uint8, device="cuda"))
    B.op_linear_q8(model(dtype="fp8"), xq, sx, wq, sw, b, y2)
    assert torch.equal(y1, y2)


# ---------------------------------------------------------------------------
# the gated sandwich norm
# ---------------------------------------------------------------------------
class Seam:
    """Seeded inputs of a norm_gate call and its values and bounds in 64 bits."""

    def __init__(self, rows, d, heads, dtype, block, groups=1, drop=(), seed=0, mean=0.0):
        rng = np.random.default_rng(seed + rows + d)
        self.m = B.model_desc(d, heads, 256, dtype, (0, d // heads // 2, d // heads // 2), block=block)
        self.om = OL.Model(d, heads, 256, (0, d // heads // 2, d // heads // 2), block=block)
        self.dt = torch.float32 if dtype == "f32" else torch.bfloat16
        rd = "f32" if dtype == "f32" else "bf16"
        self.x, self.y = (W.round_to(rng.standard_normal((rows, d)) + mean, rd) for _ in range(2))
        self.v = {"post_g": 1 + 0.2 * rng.standard_normal(d), "post_b": 0.1 * rng.standard_normal(d),
                  "pre_g": 1 + 0.2 * rng.standard_normal(d), "pre_b": 0.1 * rng.standard_normal(d),
                  "gate": rng.standard_normal((groups, d)), "scale": 0.3 + 0.05 * rng.standard_normal(d)}
        self.v = {k: None if k in drop else W.round_to(a, "f32") for k, a in self.v.items()}
        self.group = rng.integers(0, groups, rows)
        self.rms = block == "rms_swiglu"
        self.rows, self.d = rows, d

    def reference(self):
        return OL.norm_gate(self.x, self.y, self.om, self.v["post_g"], self.v["post_b"], self.v["gate"], self.v["scale"],
                            self.group, self.v["pre_g"], self.v["pre_b"])

    def noise(self, a, g, b):
        """fp32 error of Norm(a): a sum of d terms, 64 in a row in a lane and five steps across lanes, is off by
        at most (64 + 5 + 1) 2^-24 of the terms' magnitudes; it enters the mean, and halved and squared the variance."""
        c = 0.0 if self.rms else a.mean(1, keepdims=True)
        std = np.sqrt(((a - c) ** 2).mean(1, keepdims=True))
        amp = np.abs(a).mean(1, keepdims=True) / std
        n = np.abs(a - c) / std
        e = 70 * F32 * (amp + n) + 6 * F32 * (n + np.abs(a) / std)
        return np.abs(g) * e + 2 * F32 * (np.abs(g) * n + (0.0 if self.rms else np.abs(b)))

    def bounds(self, x1):
        half = F32 if self.dt == torch.float32 else BF
        k = np.ones((self.rows, self.d))
        if self.v["gate"] is not None:
            k = np.abs(self.v["gate"][self.group])
        if self.v["scale"] is not None:
            k = k * np.abs(self.v["scale"])
        post = np.abs(self.y)
        e1 = 0.0
        if self.v["post_g"] is not None:
            e1 = self.noise(self.y, self.v["post_g"], self.v["post_b"])
            post = np.abs(OL.block_norm(self.y, self.v["post_g"], self.v["post_b"], self.om))
        dx = k * (e1 + 2 * F32 * post) + F32 * np.abs(x1)
        t_x = dx + half * (np.abs(x1) + dx)
        if self.v["pre_g"] is None:
            return t_x, None
        # an error of x' enters the second norm over the row's spread, through its own element and the statistics
        std = x1.std(1, keepdims=True) if not self.rms else np.sqrt((x1 ** 2).mean(1, keepdims=True))
        c = 0.0 if self.rms else x1.mean(1, keepdims=True)
        n = np.abs(x1 - c) / std
        through = (dx + dx.mean(1, keepdims=True) + n * np.sqrt((dx ** 2).mean(1, keepdims=True))) / std
        dn = np.abs(self.v["pre_g"]) * through + self.noise(x1, self.v["pre_g"], self.v["pre_b"])
        xn = np.abs(OL.block_norm(x1, self.v["pre_g"], self.v["pre_b"], self.om))
        return t_x, (dn, dn + half * (xn + dn))

    def call(self, x_out=None, xn=None, xs=None, x=None):
        dv = {k: None if a is None else dev(a, torch.float32) for k, a in self.v.items()}
        gates = B.norm_gate_desc(**dv)
        B.op_norm_gate(self.m, gates, dev(self.x, self.dt) if x is None else x, dev(self.y, self.dt), x_out, xn, xs,
                       row_group=torch.from_numpy(self.group.astype(np.int32)).cuda())


SEAMS = [(1, 256, 4, "bf16", 1), (7, 1536, 24, "bf16", 3), (33, 512, 8, "bf16", 1), (300, 1024, 16, "bf16", 5),
         (65, 2048, 32, "bf16", 2), (19, 1280, 20, "bf16", 4), (200, 64, 4, "f32", 1), (1, 16, 1, "f32", 1),
         (9, 48, 3, "f32", 2), (130, 128, 8, "f32", 3), (31, 1024, 16, "f32", 2), (5, 640, 10, "f32", 1),
         (3, 1088, 17, "f32", 2), (2500, 768, 12, "bf16", 7)]


# rows enough for the kernel of many rows, at every number of vectors per thread and of warps per row
MANY = [(9601, 256, 4, "bf16", 3), (4802, 512, 8, "bf16", 2), (3001, 768, 12, "bf16", 1), (2501, 1024, 16, "bf16", 4),
        (1903, 1280, 20, "bf16", 2), (1301, 1536, 24, "bf16", 3), (1280, 1792, 28, "bf16", 2), (1251, 2048, 32, "bf16", 5),
        (2501, 512, 8, "f32", 2), (1301, 1024, 16, "f32", 3), (1303, 896, 14, "f32", 1),
        # fp32 rows that end inside a team's vectors, one wider than a block of few rows, one wider than a team
        (9601, 48, 3, "f32", 2), (5001, 240, 15, "f32", 3), (2501, 592, 37, "f32", 2), (1301, 1008, 63, "f32", 1),
        (700, 2064, 129, "f32", 2), (3, 4096, 64, "f32", 1), (5, 4160, 65, "f32", 2)]


@pytest.mark.parametrize("rows,d,heads,dtype,groups", SEAMS + MANY)
@pytest.mark.parametrize("block", ["ln_gelu", "rms_swiglu"])
@pytest.mark.parametrize("mean", [0.0, 4.0])
def test_norm_gate(rows, d, heads, dtype, groups, block, mean):
    c = Seam(rows, d, heads, dtype, block, groups, mean=mean)
    x_out, xn = (torch.full((rows + 1, d), 5.0, dtype=c.dt, device="cuda") for _ in range(2))
    c.call(x_out[:rows], xn[:rows])
    x1, n1 = c.reference()
    t_x, (_, t_n) = c.bounds(x1)
    assert (np.abs(host(x_out)[:rows] - x1) <= t_x).all()
    assert (np.abs(host(xn)[:rows] - n1) <= t_n).all()
    assert (host(x_out)[rows] == 5.0).all() and (host(xn)[rows] == 5.0).all()


@pytest.mark.parametrize("drop", [("gate",), ("scale",), ("gate", "scale"), ("post_g", "post_b"), ("pre_g", "pre_b"),
                                  ("post_g", "post_b", "gate", "scale", "pre_g", "pre_b")])
@pytest.mark.parametrize("rows,d,heads,dtype", [(21, 512, 8, "bf16"), (21, 48, 3, "f32"), (21, 256, 4, "f32")])
def test_norm_gate_without_a_part_and_in_place(rows, d, heads, dtype, drop):
    c = Seam(rows, d, heads, dtype, "ln_gelu", 2, drop=drop)
    if "gate" in drop:
        c.group[:] = 0
    x = dev(c.x, c.dt)
    xn = None if "pre_g" in drop else torch.empty_like(x)
    c.call(x, xn, x=x)
    x1, n1 = c.reference()
    t_x, t_n = c.bounds(x1)
    assert (np.abs(host(x) - x1) <= t_x).all()
    if xn is not None:
        assert (np.abs(host(xn) - n1) <= t_n[1]).all()


@pytest.mark.parametrize("rows,d", [(1, 256), (9, 1536), (300, 1024), (40, 2048), (9601, 256), (1301, 1536), (2501, 1024)])
@pytest.mark.parametrize("block", ["ln_gelu", "rms_swiglu"])
def test_norm_gate_int8_rows(rows, d, block):
    c = Seam(rows, d, d // 64, "int8", block, 2)
    x_out = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    xn = torch.empty((rows, d), dtype=torch.int8, device="cuda")
    xs = torch.empty(rows, device="cuda")
    c.call(x_out, xn, xs)
    x1, n1 = c.reference()
    t_x, (dn, _) = c.bounds(x1)
    assert (np.abs(host(x_out) - x1) <= t_x).all()
    top = np.abs(n1).max(1)
    s = host(xs)
    assert (np.abs(s - top / 127) <= (dn.max(1) + 2 * F32 * top) / 127).all()
    # each value lies within half a step of its integer, and its own error
    assert (np.abs(host(xn) * s[:, None] - n1) <= 0.5 * s[:, None] + dn + 4 * F32 * top[:, None]).all()
    assert (np.abs(host(xn)).max(1) == 127).all()


@pytest.mark.parametrize("rows", [50, 3001])
def test_norm_gate_e4m3_rows(rows):
    """e4m3 within half a step (2^-4) of the value of the row that is normalised in 64 bits."""
    c = Seam(rows, 768, 12, "fp8", "ln_gelu", 3)
    x_out = torch.empty((rows, 768), dtype=torch.bfloat16, device="cuda")
    xn = torch.empty((rows, 768), dtype=torch.uint8, device="cuda")
    xs = torch.empty(rows, device="cuda")
    c.call(x_out, xn, xs)
    x1, n1 = c.reference()
    _, (dn, _) = c.bounds(x1)
    v = xn.view(torch.float8_e4m3fn).double().cpu().numpy() * host(xs)[:, None]
    assert (np.abs(v - n1) <= 2.0 ** -4 * (np.abs(n1) + dn) + 2.0 ** -10 * host(xs)[:, None] + dn).all()


@pytest.mark.parametrize("rows,d,heads,dtype", [(40, 512, 8, "bf16"), (40, 48, 3, "f32"), (2501, 1024, 16, "bf16"),
                                                (40, 4160, 65, "f32")])
def test_norm_gate_group_out_of_range_is_reported_and_leaves_the_row(rows, d, heads, dtype):
    c = Seam(rows, d, heads, dtype, "ln_gelu", 3)
    c.group[[7, 31]] = [3, -1]
    x_out, xn = (torch.full((rows, d), 5.0, dtype=c.dt, device="cuda") for _ in range(2))
    c.call(x_out, xn)
    torch.cuda.synchronize()
    with pytest.raises(B.TileShareError) as e:
        B.device_status()
    assert e.value.status == 5
    B.device_status()                                  # the word is cleared
    c.group[[7, 31]] = 0
    x1, n1 = c.reference()
    t_x, (_, t_n) = c.bounds(x1)
    keep = [r for r in range(rows) if r not in (7, 31)]
    assert (np.abs(host(x_out) - x1) <= t_x)[keep].all() and (np.abs(host(xn) - n1) <= t_n)[keep].all()
    assert (host(x_out)[[7, 31]] == 5.0).all() and (host(xn)[[7, 31]] == 5.0).all()


@pytest.mark.parametrize("rows", [12, 4901])
def test_norm_gate_rows_that_are_not_finite_stay_apart(rows):
    c = Seam(rows, 512, 8, "int8", "ln_gelu", 1)
    c.y[3, 5] = np.nan
    c.x[8, 100] = np.inf
    x_out = torch.empty((rows, 512), dtype=torch.bfloat16, device="cuda")
    xn, xs = torch.empty((rows, 512), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    c.call(x_out, xn, xs)
    s = host(xs)
    assert np.isnan(s[[3, 8]]).all() and np.isfinite(np.delete(s, [3, 8])).all()
    assert (host(xn)[[3, 8]] == 0).all()


# ---------------------------------------------------------------------------
# together, as a block uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,d,N,epi", [(1, 1536, 6144, "gelu"), (21, 256, 200, "bias"), (300, 1024, 520, "swiglu")])
def test_seam_then_product(rows, d, N, epi):
    c = Seam(rows, d, d // 64, "int8", "rms_swiglu" if epi == "swiglu" else "ln_gelu", 2)
    x_out = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    xn, xs = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    rng = np.random.default_rng(3)
    wide = 2 * N if epi == "swiglu" else N
    wq = rng.integers(-127, 128, (wide, d))
    sw = np.full(wide, 2.0 ** -12)
    b = W.round_to(rng.standard_normal(wide), "f32")
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    c.call(x_out, xn, xs)
    B.op_linear_q8(c.m, xn, xs, i8(wq), dev(sw, torch.float32), dev(b, torch.float32), y, EPIS[epi])
    # the product of the rows that the norm wrote
    want, tol = linear_reference(host(xn), host(xs), wq, sw, b, epi)
    assert (np.abs(host(y) - want) <= tol).all()


def test_streams_graphs_and_repeats_agree():
    """Another stream, a captured graph replayed with new inputs in the same buffers, and a second run give the
    same bits."""
    M, K, N = 70, 512, 264
    c = Seam(M, K, 8, "int8", "ln_gelu", 2)
    rng = np.random.default_rng(0)
    wq, sw = i8(rng.integers(-127, 128, (N, K))), torch.full((N,), 2.0 ** -12, device="cuda")
    b = dev(rng.standard_normal(N), torch.float32)
    gates = B.norm_gate_desc(**{k: dev(a, torch.float32) for k, a in c.v.items()})
    group = torch.from_numpy(c.group.astype(np.int32)).cuda()
    x, y = dev(c.x, c.dt), dev(c.y, c.dt)

    def buffers():
        return dict(x1=torch.zeros_like(x), xn=torch.zeros((M, K), dtype=torch.int8, device="cuda"),
                    xs=torch.zeros(M, device="cuda"), o=torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"),
                    z=torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"),
                    sc=torch.zeros(M * K + 4 * M, dtype=torch.uint8, device="cuda"))

    def go(o, stream=None):
        B.op_norm_gate(c.m, gates, x, y, o["x1"], o["xn"], o["xs"], row_group=group, stream=stream)
        B.op_linear_q8(c.m, o["xn"], o["xs"], wq, sw, b, o["o"], B.TS_EPI_BIAS_GELU, stream=stream)
        B.op_linear(c.m, o["x1"], wq, b, o["z"], B.TS_EPI_BIAS, w_scale=sw, scratch=o["sc"], stream=stream)

    first, again, side, graphed = (buffers() for _ in range(4))
    go(first)
    go(again)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    go(side, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(graphed)
    g.replay()
    torch.cuda.synchronize()
    for o in (again, side, graphed):
        for k in ("x1", "xn", "xs", "o", "z"):
            assert torch.equal(first[k], o[k]), k
    x.copy_(dev(c.y, c.dt))
    g.replay()
    go(first)
    torch.cuda.synchronize()
    for k in ("x1", "xn", "xs", "o", "z"):
        assert torch.equal(first[k], graphed[k]), k
    assert not torch.equal(first["o"], again["o"])


def test_two_streams_at_once_agree():
    """Two calls in flight with their own buffers give what each gives alone."""
    K, N = 1024, 2048
    rng = np.random.default_rng(1)
    wq, sw = i8(rng.integers(-127, 128, (N, K))), torch.full((N,), 2.0 ** -12, device="cuda")
    b = dev(rng.standard_normal(N), torch.float32)
    m = model()
    xs = [dev(rng.standard_normal((M, K)), torch.bfloat16) for M in (4, 700)]
    alone, both = [[torch.zeros((x.shape[0], N), dtype=torch.bfloat16, device="cuda") for x in xs] for _ in range(2)]
    scratch = [torch.zeros(x.shape[0] * (K + 4), dtype=torch.uint8, device="cuda") for x in xs]
    for x, y, sc in zip(xs, alone, scratch):
        B.op_linear(m, x, wq, b, y, w_scale=sw, scratch=sc)
        torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, y, sc, s in zip(xs, both, scratch, st):
            B.op_linear(m, x, wq, b, y, w_scale=sw, scratch=sc, stream=s)
    torch.cuda.synchronize()
    for p, q in zip(alone, both):
        assert torch.equal(p, q)


# ---------------------------------------------------------------------------
# layers and the stack
# ---------------------------------------------------------------------------
SMALL = W.small_config("small_int8", d=256, heads=4, mlp=512, dtype="int8", L=3, k=1)
VOL = W.small_config("vol_int8", grid=(3, 9, 12), win=(2, 6, 8), stride=(1, 3, 4), d=256, heads=4, mlp=512, dtype="int8",
                     rope_dims=(16, 24, 24))
RMS = dataclasses.replace(SMALL, name="rms_int8", block="rms_swiglu")
# Two bf16-level paths differ by up to 1e-2 (the bf16 suite's bound).  With integers a value x off by up to half a
# bf16 step (2^-9 of it in the mean) may fall on the other side of a border between two steps of a / 127, a about 4
# deviations: rms sqrt(4/127 * 2^-10) = 0.6 % of the row for each of four GEMMs, 1.1 % together on the branch.
TOL = {"f32": 1e-5, "bf16": 1e-2, "fp8": 3e-2, "int8": 2e-2}


def layer_on_device(cfg, p):
    out = {}
    for k, v in p.items():
        if k not in BIG:
            out[k] = dev(v, torch.float32)
            continue
        t = dev(v, torch.float32 if cfg.dtype == "f32" else torch.bfloat16)
        if cfg.dtype in ("fp8", "int8"):
            q = torch.empty(t.shape, dtype=torch.uint8, device="cuda")
            s = torch.empty(t.shape[0], device="cuda")
            (B.quantize_rows_i8 if cfg.dtype == "int8" else B.quantize_rows_e4m3)(t, q, s)
            out[k], out[SCALE[k]] = q, s
        else:
            out[k] = t
    return out


class Layers:
    def __init__(self, cfg, seed=0):
        self.cfg = cfg
        self.op = OP.make_plan(cfg.grid, cfg.win, cfg.stride, registers=cfg.R)
        self.plan = B.Plan(cfg.grid, cfg.win, cfg.stride, registers=cfg.R)
        dr = W.Draw(cfg, self.op.T, seed=seed, affine=True)
        self.S0, self.G0 = dr.states()
        self.p = dr.layers()
        self.m = B.model_desc(cfg.d, cfg.heads, cfg.mlp, cfg.dtype, cfg.rope_dims, block=cfg.block)
        self.om = OL.Model(cfg.d, cfg.heads, cfg.mlp, cfg.rope_dims, fp8=cfg.dtype == "fp8", int8=cfg.dtype == "int8",
                           block=cfg.block)
        self.w = [B.layer_weights(layer_on_device(cfg, p)) for p in self.p]
        self.dt = torch.float32 if cfg.dtype == "f32" else torch.bfloat16
        self.S = np.concatenate([self.S0, self.G0])

    def ws(self, L=0, k=0):
        return torch.empty(B.workspace_size(self.plan, self.m, L, k), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("cfg", [SMALL, VOL, RMS], ids=lambda c: c.name)
def test_int8_layers(cfg):
    c = Layers(cfg)
    S = dev(c.S, c.dt)
    B.block_shared(c.plan, c.m, c.w[0], S, c.ws())
    want = OL.block_shared(c.S, c.p[0], c.om, c.op)
    assert rel_l2(host(S), want) < TOL["int8"]
    assert_rows(host(S), want, c.op, "shared", TOL["int8"])
    X0 = OL.gather(c.S, c.op)
    X = dev(X0.reshape(-1, cfg.d), c.dt)
    B.block_tiled(c.plan, c.m, c.w[0], X, c.ws())
    want = OL.block_tiled(X0, c.p[0], c.om, c.op).reshape(-1, cfg.d)
    assert rel_l2(host(X), want) < TOL["int8"]
    if cfg is SMALL:
        X = dev(X0.reshape(-1, cfg.d), c.dt)
        B.block_partial(c.plan, c.m, c.w[0], B.TS_SHARE_QKV | B.TS_SHARE_MLP, X, c.ws())
        want = OL.block_partial(X0, c.p[0], c.om, c.op, ("qkv", "mlp")).reshape(-1, cfg.d)
        assert rel_l2(host(X), want) < TOL["int8"]
        S1, S2 = dev(c.S, c.dt), dev(c.S, c.dt)
        B.block_shared(c.plan, c.m, c.w[0], S1, c.ws())
        B.block_shared_noalloc(c.plan, c.m, c.w[0], S2)
        assert torch.equal(S1, S2)


@pytest.mark.parametrize("k", [0, 1, 3])
def test_int8_stack(k):
    c = Layers(SMALL)
    out = torch.empty((c.op.U, SMALL.d), dtype=c.dt, device="cuda")
    B.decode_stack(c.plan, c.m, c.w, k, dev(c.S0, c.dt), dev(c.G0, c.dt), out, c.ws(3, k))
    want = OL.decode_stack(c.S0, c.G0, c.p, c.om, c.op, k)
    assert rel_l2(host(out), want) < TOL["int8"]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("block", ["ln_gelu", "rms_swiglu"])
@pytest.mark.parametrize("parts", ["all", "gates", "norms", "none"])
def test_sandwich_layers(dtype, block, parts):
    cfg = dataclasses.replace(SMALL, name="sandwich", dtype=dtype, block=block, d=64 if dtype == "f32" else 256,
                              rope_dims=(0, 8, 8) if dtype == "f32" else (0, 32, 32), R=2)
    c = Layers(cfg)
    rng = np.random.default_rng(4)
    vec = {}
    for i in (1, 2):
        if parts in ("all", "norms"):
            vec[f"post{i}_g"] = 1 + 0.2 * rng.standard_normal(cfg.d)
            vec[f"post{i}_b"] = 0.1 * rng.standard_normal(cfg.d)
        if parts in ("all", "gates"):
            vec[f"gate{i}"] = 0.5 * rng.standard_normal((3, cfg.d))
            vec[f"scale{i}"] = 0.7 + 0.1 * rng.standard_normal(cfg.d)
    vec = {k: W.round_to(v, "f32") for k, v in vec.items()}
    for tiled in (False, True):
        state = OL.gather(c.S, c.op) if tiled else c.S
        rows = state.reshape(-1, cfg.d).shape[0]
        group = rng.integers(0, 3, rows)
        sw = B.sandwich_weights(row_group=torch.from_numpy(group.astype(np.int32)).cuda(),
                                **{k: dev(v, torch.float32) for k, v in vec.items()})
        t = dev(state.reshape(-1, cfg.d), c.dt)
        fn, ref = ((B.block_tiled_sandwich, OL.block_tiled_sandwich) if tiled else
                   (B.block_shared_sandwich, OL.block_shared_sandwich))
        with pytest.raises(B.TileShareError):
            fn(c.plan, c.m, c.w[0], B.sandwich_weights(row_group=sw._tensors["row_group"][1:]), t, c.ws())
        with pytest.raises(B.TileShareError):
            fn(c.plan, c.m, c.w[0], B.sandwich_weights(scale1=torch.ones(2 * cfg.d, device="cuda")), t, c.ws())
        fn(c.plan, c.m, c.w[0], sw, t, c.ws())
        want = ref(state, c.p[0], dict(vec, row_group=group), c.om, c.op).reshape(-1, cfg.d)
        assert rel_l2(host(t), want) < TOL[dtype]


# ---------------------------------------------------------------------------
# refusals that need device tensors
# ---------------------------------------------------------------------------
def test_binding_refuses_tensors_that_do_not_fit():
    M, K, N = 8, 128, 64
    x = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    s, b = torch.ones(N, device="cuda"), torch.zeros(N, device="cuda")
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    xb = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    scratch = torch.zeros(M * (K + 4), dtype=torch.uint8, device="cuda")
    ok = dict(model=model(), x=x, x_scale=s, W=w, w_scale=s, bias=b, y=y)
    B.op_linear_q8(**ok)
    wide = torch.zeros((M, 2 * K), dtype=torch.int8, device="cuda")
    for bad in ({"x": wide[:, :K]}, {"x": x[::2].t().contiguous()[:, :4]}, {"W": w.t()}, {"W": w[:, :64]}, {"x": x.cpu()},
                {"x": xb}, {"y": y.float()}, {"y": y[: M - 1]}, {"bias": b[: N - 1]}, {"w_scale": s[:8]},
                {"x_scale": s[: M - 1]}, {"W": w.bfloat16()}, {"y": y.t()}, {"bias": b.cpu()}, {"w_scale": s.cpu()},
                {"x_scale": s.cpu()}, {"W": w.cpu()}, {"y": y.cpu()}):
        with pytest.raises(B.TileShareError) as e:
            B.op_linear_q8(**dict(ok, **bad))
        assert e.value.status == 1
    lin = dict(model=model(), x=xb, W=w, bias=b, y=y, w_scale=s, scratch=scratch)
    B.op_linear(**lin)
    for bad in ({"x": x}, {"scratch": scratch[:-1]}, {"scratch": None}, {"w_scale": None}, {"W": w[:, ::2]}, {"x": xb[:, ::2]},
                {"scratch": scratch.cpu()}, {"bias": b.cpu()}):
        with pytest.raises(B.TileShareError) as e:
            B.op_linear(**dict(lin, **bad))
        assert e.value.status == 1
    c = Seam(M, 256, 4, "bf16", "ln_gelu", 1)
    x1 = torch.empty((M, 256), dtype=torch.bfloat16, device="cuda")
    for out in (x1.t(), x1[:-1], x1.float(), x1.cpu(), x1.to(torch.int8)):
        with pytest.raises(B.TileShareError):
            c.call(out, x1)
    with pytest.raises(B.TileShareError):
        c.call(x1, x1.to(torch.int8))                      # 8-bit rows need their scales
    with pytest.raises(B.TileShareError):                  # vectors of another width
        B.op_norm_gate(c.m, B.norm_gate_desc(scale=torch.ones(128, device="cuda")), x1, x1, x1)
    for bad in ({"gates": B.norm_gate_desc(scale=torch.ones(256))}, {"y": x1.cpu()},
                {"row_group": torch.zeros(M, dtype=torch.int32)}, {"row_group": torch.zeros(M, dtype=torch.int64, device="cuda")}):
        with pytest.raises(B.TileShareError):
            B.op_norm_gate(**dict(dict(model=c.m, gates=B.norm_gate_desc(), x=x1, y=x1, x_out=x1), **bad))
    with pytest.raises(ValueError):
        B.norm_gate_desc(scale=torch.ones(256), gate=torch.ones((1, 256), device="cuda"))
    q = torch.empty((M, K), dtype=torch.int8, device="cuda")
    for args in ((xb, q[:-1], s), (xb.t(), q, s), (xb.float(), q, s), (xb, q, s[:4])):
        with pytest.raises(B.TileShareError):
            B.quantize_rows_i8(*args)


def test_calls_with_no_rows_do_nothing():
    w, s = torch.zeros((64, 128), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    none = lambda d, t: torch.empty((0, d), dtype=t, device="cuda")   # noqa: E731
    n = B.launch_count()
    B.op_linear_q8(model(), none(128, torch.int8), s[:0], w, s, s, none(64, torch.bfloat16))
    B.op_linear(model(), none(128, torch.bfloat16), w, s, none(64, torch.bfloat16), w_scale=s, scratch=s)
    B.quantize_rows_i8(none(128, torch.bfloat16), none(128, torch.int8), s[:0])
    x = none(256, torch.bfloat16)
    B.op_norm_gate(model(), B.norm_gate_desc(), x, x, x)
    assert B.launch_count() == n


# ---------------------------------------------------------------------------
# calls that come first, large offsets, threads
# ---------------------------------------------------------------------------
FIRST_CAPTURE = '''
import numpy as np, torch
from shared_token_transformer_b200 import binding as B
m = B.model_desc(256, 4, 256, "int8", (0, 32, 32))
def call(M, K, N):
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((N, K), dtype=torch.int8, device="cuda")
    s, b = torch.full((N,), 1.0 / 127, device="cuda"), torch.zeros(N, device="cuda")
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    sc = torch.zeros(M * (K + 4), dtype=torch.uint8, device="cuda")
    return (lambda: B.op_linear(m, x, w, b, y, w_scale=s, scratch=sc)), y, K / 127, (x, w, s, b, y, sc)
def seam(M):
    x = torch.ones((M, 256), dtype=torch.bfloat16, device="cuda")
    o, g = torch.zeros_like(x), B.norm_gate_desc(scale=torch.full((256,), 2.0, device="cuda"))
    return (lambda: B.op_norm_gate(m, g, x, x, o)), o, 3.0, (x, o, g)
# one row (blocks quantise), few rows, a cluster that shares K, whole tiles, pairs of SMs; few and many rows of the seam
calls = [call(1, 256, 64), call(20, 256, 64), call(128, 2048, 128), call(2500, 256, 256), call(6000, 512, 2048), seam(3), seam(9601)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for f, *_ in calls:
        f()
g.replay()
torch.cuda.synchronize()
B.device_status()
for f, y, want, _ in calls:
    assert (y.double() - want).abs().max().item() <= want * 2.0 ** -8, (y.shape, want, y.flatten()[:4])
print("captured first")
'''


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, (r.stdout, r.stderr[-2000:])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows of the quantiser, the seam and the product are those of a small call."""
    d, rows, tail = 1024, (1 << 21) + 37, 70
    rng = np.random.default_rng(2)
    c = Seam(tail, d, 16, "int8", "ln_gelu", 1)
    x, y = (torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-tail:], y[-tail:] = dev(c.x, c.dt), dev(c.y, c.dt)
    gates = B.norm_gate_desc(**{k: dev(a, torch.float32) for k, a in c.v.items()})
    xn, xs = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    small_n, small_s = torch.empty((tail, d), dtype=torch.int8, device="cuda"), torch.empty(tail, device="cuda")
    small_x = torch.empty((tail, d), dtype=torch.bfloat16, device="cuda")
    B.op_norm_gate(c.m, gates, x, y, x, xn, xs)
    B.op_norm_gate(c.m, gates, dev(c.x, c.dt), dev(c.y, c.dt), small_x, small_n, small_s)
    # the two kernels sum in different orders: x' within a bf16 step, integers within one
    assert ((x[-tail:] - small_x).abs() <= 2.0 ** -7 * small_x.abs() + 1e-6).all()
    assert ((xn[-tail:].int() - small_n.int()).abs() <= 1).all()
    assert torch.allclose(xs[-tail:], small_s, rtol=1e-4, atol=0)
    q, s = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    B.quantize_rows_i8(x, q, s)
    want_q, want_s = I8.quantize_rows(host(x[-tail:]))
    np.testing.assert_array_equal(host(q[-tail:]), want_q)
    np.testing.assert_array_equal(host(s[-tail:]), want_s)
    del x, y, xn
    N = 1032
    wq, sw, b = i8(rng.integers(-127, 128, (N, d))), torch.full((N,), 2.0 ** -12, device="cuda"), torch.zeros(N, device="cuda")
    out, small = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda"), torch.empty((tail, N), dtype=torch.bfloat16, device="cuda")
    B.op_linear_q8(model(), q, s, wq, sw, b, out)
    B.op_linear_q8(model(), q[-tail:].clone(), s[-tail:].clone(), wq, sw, b, small)
    assert torch.equal(out[-tail:], small)


def test_host_threads_at_once_agree():
    """Two host threads on streams of their own, each with its own buffers."""
    import threading
    rng = np.random.default_rng(9)
    K, N = 512, 520
    wq, sw, b = i8(rng.integers(-127, 128, (N, K))), torch.full((N,), 2.0 ** -12, device="cuda"), torch.zeros(N, device="cuda")
    xs = [dev(rng.standard_normal((M, K)), torch.bfloat16) for M in (3, 130)]
    want = []
    for x in xs:
        y = torch.empty((x.shape[0], N), dtype=torch.bfloat16, device="cuda")
        B.op_linear(model(), x, wq, b, y, w_scale=sw, scratch=torch.empty(x.shape[0] * (K + 4), dtype=torch.uint8, device="cuda"))
        want.append(y)
    torch.cuda.synchronize()
    got, errors = [torch.zeros_like(y) for y in want], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            scratch = torch.empty(xs[i].shape[0] * (K + 4), dtype=torch.uint8, device="cuda")
            for _ in range(100):
                B.op_linear(model(), xs[i], wq, b, got[i], w_scale=sw, scratch=scratch, stream=s)
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(torch.equal(a, w) for a, w in zip(got, want))


@pytest.mark.parametrize("mode", [B.TS_ROWS_SHARED, B.TS_ROWS_TILED])
def test_int8_qkv_values(mode):
    """The v part of op_qkv is the int8 linear layer of Norm1 (q and k pass the norm and rotation of every dtype)."""
    c = Layers(SMALL)
    state = c.S if mode == B.TS_ROWS_SHARED else OL.gather(c.S, c.op).reshape(-1, SMALL.d)
    rows, d = state.shape
    qkv = torch.empty((rows, 3 * d), dtype=torch.bfloat16, device="cuda")
    B.op_qkv(c.plan, c.m, c.w[0], mode, dev(state, c.dt), qkv, torch.empty(rows * d * 6 + 8192, dtype=torch.uint8, device="cuda"))
    q, k, v = OL.qkv_project(state, c.p[0], c.om)
    assert rel_l2(host(qkv)[:, 2 * d:], v.reshape(rows, d)) < TOL["int8"]
    # rotation keeps each head's norm
    for part, want in ((0, q), (1, k)):
        got = host(qkv)[:, part * d:(part + 1) * d].reshape(rows, SMALL.heads, -1)
        assert rel_l2(np.linalg.norm(got, axis=2), np.linalg.norm(want, axis=2)) < TOL["int8"]
