"""Timed cases of the 8-bit integer linear layer and of the gated sandwich norm.

linear       y = act((q(x) W8^T) * sx * sw + b), x bf16 quantised per token inside the call
linear_q8    the same product of rows that are 8-bit integers with scales already
norm_gate    x' = x + gate * scale * Norm(y); xn = Norm(x')
norm_linear  norm_gate handing 8-bit rows to linear_q8: the seam between two halves of a block

Sizes are those of the package's workloads (d 512, 1024, 1536; MLP 2048, 4096, 6144; 48x48, 128x128,
256x256 and 4x44x80 tokens with one register row per tile), with single rows and ragged sizes beside them.
"""

import functools
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
TINY = 2.0 ** -100      # rows whose largest magnitude is below this count as zero


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _linear(name, rows, K, N, epi, op="linear"):
    return {"name": name, "op": op, "rows": rows, "K": K, "N": N, "epi": epi}


def _norm(name, rows, d, heads, dtype, norm, groups):
    return {"name": name, "op": "norm_gate", "rows": rows, "d": d, "heads": heads, "dtype": dtype, "norm": norm,
            "groups": groups}


def _seam(name, rows, d, N, epi, norm, groups):
    return {"name": name, "op": "norm_linear", "rows": rows, "d": d, "N": N, "epi": epi, "norm": norm,
            "groups": groups}


def listed():
    return [
        # one token through the video decoder's QKV projection: latency
        _linear("token_qkv", 1, 1536, 4608, "bias"),
        # the register rows of the video grid's six tiles through the MLP down projection
        _linear("registers_down", 6, 6144, 1536, "bias"),
        # a ragged projection between models: odd rows, K and N off every tile size
        _linear("ragged", 333, 1040, 1336, "bias"),
        # 48x48 tokens and 16 register rows, MLP up
        _linear("stack48_up", 2320, 512, 2048, "gelu"),
        # 2K image (128x128 tokens, 25 tiles), MLP up
        _linear("image2k_up", 16409, 1024, 4096, "gelu"),
        # 4K image (256x256 tokens, 121 tiles), SwiGLU MLP up: the largest
        _linear("image4k_swiglu", 65657, 1024, 4096, "swiglu"),
        # video QKV projection of rows that the norm has quantised
        _linear("video_qkv_q8", 14086, 1536, 4608, "bias", "linear_q8"),
        # a tile's worth of quantised rows, MLP down of the 2K image model
        _linear("tile_down_q8", 257, 4096, 1024, "bias", "linear_q8"),
        # the video state, one gate per latent frame, LayerNorm on both sides
        _norm("video_norm", 14086, 1536, 24, "bf16", "ln", 4),
        # the fp32 14x14 block with four tiles' registers, RMSNorm
        _norm("vit14_norm_f32", 200, 64, 4, "f32", "rms", 1),
        # the seam attention -> MLP for one token
        _seam("token_seam", 1, 1536, 6144, "gelu", "ln", 1),
        # the same seam for the 2K image, RMSNorm and SwiGLU
        _seam("image2k_seam", 16409, 1024, 4096, "swiglu", "rms", 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["linear", "linear", "linear_q8", "norm_gate", "norm_linear"])
        rows = _log(rng, 1, 65657)
        epi = rng.choice(["bias", "gelu", "swiglu"])
        norm = rng.choice(["ln", "rms"])
        if op in ("linear", "linear_q8"):
            c = {"op": op, "rows": rows, "K": 16 * _log(rng, 4, 512), "N": 8 * _log(rng, 8, 1024), "epi": epi}
        elif op == "norm_gate":
            if rng.random() < 0.25:
                heads = rng.randint(1, 16)
                c = {"op": op, "rows": rows, "d": heads * rng.choice([16, 32, 64]), "heads": heads, "dtype": "f32"}
            else:
                d = 256 * rng.randint(1, 8)
                c = {"op": op, "rows": rows, "d": d, "heads": d // 64, "dtype": "bf16"}
            c.update(norm=norm, groups=rng.randint(1, 8))
        else:
            c = {"op": op, "rows": rows, "d": 256 * rng.randint(1, 8), "N": 8 * _log(rng, 8, 1024), "epi": epi,
                 "norm": norm, "groups": rng.randint(1, 8)}
        if _cost(c) <= most:
            return c


def work(case):
    """Bytes that must be read and written once, and operations of the products."""
    m = case["rows"]
    if case["op"] == "norm_gate":
        e, d = DT[case["dtype"]].itemsize, case["d"]
        return {"bytes": 4 * m * d * e + 4 * m + 4 * d * (case["groups"] + 5), "flops": 30 * m * d}
    wide = 2 * case["N"] if case["epi"] == "swiglu" else case["N"]
    if case["op"] == "norm_linear":
        k = case["d"]
        read = 4 * m * k + 2 * m * k + 4 * m + 4 * k * (case["groups"] + 5)     # x, y in; x' out; groups; vectors
    else:
        k = case["K"]
        read = 2 * m * k if case["op"] == "linear" else m * k + 4 * m
    return {"bytes": read + wide * k + 8 * wide + 2 * m * case["N"], "flops": 2 * m * wide * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * std + mean

    def activations(rows, cols, dtype):
        # a few channels carry large values, as the residual stream of trained transformers has them
        gain = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        return (normal(rows, cols) * gain).to(dtype)

    m, op = case["rows"], case["op"]
    st = {"case": case}
    k = case.get("K", case.get("d"))
    if op in ("linear", "linear_q8", "norm_linear"):
        n = case["N"]
        wide = 2 * n if case["epi"] == "swiglu" else n
        st["w"], st["w_scale"] = _quantise(normal(wide, k, std=0.02).to(torch.bfloat16))
        st["bias"] = normal(wide, std=0.1)
        st["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    if op == "linear":
        st["x"] = activations(m, k, torch.bfloat16)
        st["scratch"] = torch.empty(m * k + 4 * m, dtype=torch.uint8, device="cuda")
    elif op == "linear_q8":
        st["x"], st["x_scale"] = _quantise(activations(m, k, torch.bfloat16))
    else:
        dt = DT[case.get("dtype", "bf16")]
        st["x"] = activations(m, k, dt)          # the residual stream
        st["y"] = activations(m, k, dt)          # the block's output
        st["post_g"], st["post_b"] = normal(k, std=0.2, mean=1.0), normal(k, std=0.1)
        st["pre_g"], st["pre_b"] = normal(k, std=0.2, mean=1.0), normal(k, std=0.1)
        st["scale"] = normal(k, std=0.05, mean=0.3)
        st["gate"] = normal(case["groups"], k, std=0.5)
        st["row_group"] = (torch.arange(m, device="cuda") * case["groups"] // m).to(torch.int32)   # frame by frame
        st["x_out"] = torch.empty_like(st["x"])
        if op == "norm_gate":
            st["xn"] = torch.empty_like(st["x"])
        else:
            st["xn"] = torch.empty(m, k, dtype=torch.int8, device="cuda")
            st["xn_scale"] = torch.empty(m, dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _quantise(x):
    """Rows as 8-bit integers with one fp32 scale each: inv = 127 / max|x| rounded to fp32, q the integer
    nearest to x * inv (in 64 bits: values next to a border), scale = max|x| / 127."""
    x = x.float()
    top = x.abs().amax(dim=1)
    none = top < TINY
    safe = torch.where(none, torch.ones_like(top), top)
    steps = torch.full_like(top, 127.0)      # tensor by tensor: a scalar operand would go through a reciprocal
    inv = torch.where(none, torch.zeros_like(top), steps / safe)
    scale = torch.where(none, torch.ones_like(top), safe / steps)
    q = torch.round(x.double() * inv.double()[:, None])
    return q.to(torch.int8), scale


def _activation(acc, epi):
    if epi == "gelu":
        return 0.5 * acc * (1.0 + torch.erf(acc * (0.5 ** 0.5)))
    if epi == "swiglu":
        n = acc.shape[1] // 2
        gate, up = acc[:, :n], acc[:, n:]
        return gate / (1.0 + torch.exp(-gate)) * up
    return acc


def _product(q, scale, st):
    acc = q.float() @ st["w"].float().t()
    acc = acc * scale[:, None] * st["w_scale"][None, :] + st["bias"][None, :]
    return _activation(acc, st["case"]["epi"]).to(torch.bfloat16)


def _normed(v, gain, bias, kind):
    if kind == "rms":
        return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * gain
    c = v - v.mean(dim=1, keepdim=True)
    return c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) * gain + bias


def _joined(st):
    kind = st["case"]["norm"]
    post = _normed(st["y"].float(), st["post_g"], st["post_b"], kind)
    x = st["x"].float() + st["gate"][st["row_group"].long()] * st["scale"] * post
    return x, _normed(x, st["pre_g"], st["pre_b"], kind)


def _plain(st):
    op = st["case"]["op"]
    if op == "linear":
        return _product(*_quantise(st["x"]), st)
    if op == "linear_q8":
        return _product(st["x"], st["x_scale"], st)
    x, xn = _joined(st)
    if op == "norm_gate":
        return {"x_out": x.to(st["x"].dtype), "xn": xn.to(st["x"].dtype)}
    return {"x_out": x.to(st["x"].dtype), "out": _product(*_quantise(xn), st)}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _model(d, heads, dtype, block):
    from shared_token_transformer_b200 import binding as B
    hd = d // heads
    return B.model_desc(d, heads, 4 * d, dtype, (0, hd // 2, hd // 2), eps_ln=EPS, block=block)


def _framework(st):
    from shared_token_transformer_b200 import binding as B
    c = st["case"]
    op = c["op"]
    if op != "norm_gate":
        epi = {"bias": B.TS_EPI_BIAS, "gelu": B.TS_EPI_BIAS_GELU, "swiglu": B.TS_EPI_BIAS_SWIGLU}[c["epi"]]
    if op == "linear":
        B.op_linear(_model(1024, 16, "int8", "ln_gelu"), st["x"], st["w"], st["bias"], st["out"], epi,
                    w_scale=st["w_scale"], scratch=st["scratch"])
        return st["out"]
    if op == "linear_q8":
        B.op_linear_q8(_model(1024, 16, "int8", "ln_gelu"), st["x"], st["x_scale"], st["w"], st["w_scale"], st["bias"],
                       st["out"], epi)
        return st["out"]
    block = "rms_swiglu" if c["norm"] == "rms" else "ln_gelu"
    if "gates" not in st:      # the descriptor that a program keeps beside its weights
        st["gates"] = B.norm_gate_desc(post_g=st["post_g"], post_b=st["post_b"], pre_g=st["pre_g"], pre_b=st["pre_b"],
                                       gate=st["gate"], scale=st["scale"])
    if op == "norm_gate":
        B.op_norm_gate(_model(c["d"], c["heads"], c["dtype"], block), st["gates"], st["x"], st["y"], st["x_out"],
                       st["xn"], row_group=st["row_group"])
        return {"x_out": st["x_out"], "xn": st["xn"]}
    model = _model(c["d"], c["d"] // 64, "int8", block)
    B.op_norm_gate(model, st["gates"], st["x"], st["y"], st["x_out"], st["xn"], xn_scale=st["xn_scale"],
                   row_group=st["row_group"])
    B.op_linear_q8(model, st["xn"], st["xn_scale"], st["w"], st["w_scale"], st["bias"], st["out"], epi)
    return {"x_out": st["x_out"], "out": st["out"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(x64):
    """Integers and scales of rows given in 64 bits; the reciprocal 127 / max|x| is an fp32 number by definition."""
    top = x64.abs().max(dim=1, keepdim=True).values
    empty = top < TINY
    steps = torch.full_like(top, 127.0)
    inv = (steps / top.clamp_min(TINY)).float().double().masked_fill(empty, 0.0)
    scale = (top / steps).float().double().masked_fill(empty, 1.0)
    return (x64 * inv).round(), scale


def _exact_linear(q, scale, st):
    z = torch.matmul(q, st["w"].double().transpose(0, 1)).mul_(scale).mul_(st["w_scale"].double())
    z += st["bias"].double()
    epi, n = st["case"]["epi"], st["case"]["N"]
    if epi == "gelu":
        return z * torch.special.ndtr(z)
    if epi == "swiglu":
        return z[:, :n] * torch.sigmoid(z[:, :n]) * z[:, n:]
    return z


def _exact_norm(v, gain, bias, kind):
    mean = torch.zeros_like(v[:, :1]) if kind == "rms" else v.mean(dim=1, keepdim=True)
    spread = torch.sqrt(((v - mean) ** 2).mean(dim=1, keepdim=True) + EPS)
    out = (v - mean) / spread * gain.double()
    return out if kind == "rms" else out + bias.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(*_exact_rows(st["x"].double()), st)
    if op == "linear_q8":
        return _exact_linear(st["x"].double(), st["x_scale"].double()[:, None], st)
    branch = _exact_norm(st["y"].double(), st["post_g"], st["post_b"], case["norm"])
    x = st["x"].double() + st["gate"].double()[st["row_group"].long()] * st["scale"].double() * branch
    xn = _exact_norm(x, st["pre_g"], st["pre_b"], case["norm"])
    if op == "norm_gate":
        return {"x_out": x, "xn": xn}
    return {"x_out": x, "out": _exact_linear(*_exact_rows(xn), st)}
