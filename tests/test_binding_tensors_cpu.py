"""Which tensors the 8-bit and seam calls of the binding take: checked on host tensors, with a
library that records calls in place of the built one, so that nothing reaches a device."""

import pytest
import torch

from shared_token_transformer_b200 import binding as B
from shared_token_transformer_b200 import build as Bd


# ---------------------------------------------------------------------------
# descriptors of norms, gates and scales
# ---------------------------------------------------------------------------
def test_a_gate_given_as_a_vector_is_one_group():
    """The kernel holds each row's group against `groups`; every group it lets through must lie in the gate."""
    assert B.norm_gate_desc(gate=torch.zeros(64), scale=torch.zeros(64)).groups == 1
    assert B.norm_gate_desc(gate=torch.zeros(3, 64)).groups == 3
    sw = B.sandwich_weights(gate1=torch.zeros(1, 64), gate2=torch.zeros(64))
    assert (sw.groups, sw.width) == (1, 64)
    with pytest.raises(ValueError):
        B.sandwich_weights(gate1=torch.zeros(64), gate2=torch.zeros(64, 64))


@pytest.mark.parametrize("name", ["post_g", "post_b", "pre_g", "pre_b", "gate", "scale"])
def test_vectors_are_fp32(name):
    for dtype in (torch.int32, torch.uint32, torch.float64, torch.bfloat16):
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(2, 64).to(dtype)})


def test_row_groups_of_a_sandwich_are_int32():
    for dtype in (torch.float32, torch.uint32, torch.int64):
        with pytest.raises(ValueError):
            B.sandwich_weights(row_group=torch.zeros(8).to(dtype))
    with pytest.raises(ValueError):
        B.sandwich_weights(row_group=torch.zeros(16, dtype=torch.int32)[::2])
    assert B.sandwich_weights(row_group=torch.zeros(8, dtype=torch.int32)).row_group


@pytest.mark.parametrize("name", ["post_g", "post_b", "pre_g", "pre_b", "gate", "scale"])
def test_vectors_are_single_and_not_empty(name):
    for shape in ((0,), (0, 64), (2, 0), ()):      # the address of nothing would read as "none"
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(shape)})
    assert getattr(B.norm_gate_desc(**{name: torch.zeros(1, 64)}), name)
    if name != "gate":                             # rows past the first would be left out
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(2, 64)})


# ---------------------------------------------------------------------------
# tensors of the calls
# ---------------------------------------------------------------------------
BF, F32, I8, U8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.uint8, torch.int32
ROWS, K, N = 6, 256, 64


@pytest.fixture
def calls(monkeypatch):
    """Host tensors count as those of the current device, and the library notes the names of its calls."""
    class Library:
        def __init__(self):
            self.names = []

        def __getattr__(self, name):
            return lambda *a: self.names.append(name) or 0

    L = Library()
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(B, "_lib", L)
    monkeypatch.setattr(B, "_device", None)
    monkeypatch.setattr(B, "_raw_stream", None)
    return L.names


def model(dtype="int8"):
    return B.model_desc(K, 4, 256, dtype, (0, 32, 32))


def z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "quantize": (B.quantize_rows_i8, lambda: dict(x=z(ROWS, K, dtype=BF), q=z(ROWS, K, dtype=I8), scale=z(ROWS))),
    "linear": (B.op_linear, lambda: dict(model=model(), x=z(ROWS, K, dtype=BF), W=z(N, K, dtype=I8), bias=z(N),
                                         y=z(ROWS, N, dtype=BF), w_scale=z(N),
                                         scratch=z(ROWS * (K + 4), dtype=U8))),
    "linear_q8": (B.op_linear_q8, lambda: dict(model=model(), x=z(ROWS, K, dtype=I8), x_scale=z(ROWS),
                                               W=z(N, K, dtype=I8), w_scale=z(N), bias=z(N), y=z(ROWS, N, dtype=BF))),
    "norm_gate": (B.op_norm_gate, lambda: dict(model=model(), gates=B.norm_gate_desc(gate=z(3, K), pre_g=z(K), pre_b=z(K)),
                                               x=z(ROWS, K, dtype=BF), y=z(ROWS, K, dtype=BF), x_out=z(ROWS, K, dtype=BF),
                                               xn=z(ROWS, K, dtype=I8), xn_scale=z(ROWS), row_group=z(ROWS, dtype=I32))),
}
TENSORS = [(c, n) for c, (_, make) in CALLS.items() for n, v in make().items() if isinstance(v, torch.Tensor)]


def refused(calls, name, **bad):
    fn, make = CALLS[name]
    calls.clear()
    with pytest.raises(B.TileShareError) as e:
        fn(**dict(make(), **bad))
    assert e.value.status == 1 and not calls


@pytest.mark.parametrize("name", CALLS)
def test_tensors_that_fit_are_taken(calls, name):
    fn, make = CALLS[name]
    fn(**make())
    # outputs and vectors may be longer than the call needs
    for n, longer in (("q", z(ROWS + 1, K, dtype=I8)), ("scale", z(ROWS + 3)), ("y", z(ROWS + 2, N, dtype=BF)),
                      ("bias", z(N + 8)), ("w_scale", z(N + 8)), ("x_scale", z(ROWS + 1)), ("scratch", z(3 * K * ROWS, dtype=U8)),
                      ("x_out", z(ROWS + 1, K, dtype=BF)), ("xn", z(ROWS + 1, K, dtype=I8)), ("xn_scale", z(ROWS + 1)),
                      ("q", z(ROWS * K, dtype=I8)), ("W", z(N, K, dtype=U8))):
        if n in make() and not (n == "y" and name == "norm_gate"):
            fn(**dict(make(), **{n: longer}))
    assert len(calls) > 1


@pytest.mark.parametrize("name,tensor", TENSORS)
def test_strided_and_expanded_tensors_are_refused(calls, name, tensor):
    """An expanded tensor counts bytes that it does not have; the elements of a strided one lie elsewhere."""
    t = CALLS[name][1]()[tensor]
    refused(calls, name, **{tensor: torch.zeros((1,) * t.dim(), dtype=t.dtype).expand(t.shape)})
    every_second = torch.zeros((*t.shape, 2), dtype=t.dtype)[..., 0]
    assert every_second.shape == t.shape
    refused(calls, name, **{tensor: every_second})


@pytest.mark.parametrize("name,tensor", [t for t in TENSORS if t[1] != "scratch"])
def test_other_element_types_are_refused(calls, name, tensor):
    """Also those of the same size: their bits would be read as the type of the call."""
    t = CALLS[name][1]()[tensor]
    same = {1: (torch.bool, torch.float8_e4m3fn, torch.float8_e5m2), 2: (torch.float16, torch.int16),
            4: (torch.int32, torch.float32, torch.uint32)}[t.element_size()]
    for dtype in (*same, torch.float64, torch.int64):
        if dtype is not t.dtype:
            refused(calls, name, **{tensor: torch.zeros(t.shape, dtype=torch.uint8).to(dtype)})
    # as many bytes of a type twice as wide
    refused(calls, name, **{tensor: torch.zeros(t.numel() // 2, dtype=torch.float64).reshape(-1, *t.shape[1:])
                            if t.dim() == 1 else torch.zeros((t.shape[0], t.shape[1] // 2), dtype=torch.float64)})


def test_types_of_8_bit_rows_belong_to_the_model(calls):
    """Bytes as the quantisers fill them, or the type that the model computes in."""
    fn, make = CALLS["linear_q8"]
    e4m3, i8, u8 = (lambda n, t=t: z(n, K, dtype=t) for t in (torch.float8_e4m3fn, I8, U8))
    for dtype, own, other in (("int8", i8, e4m3), ("fp8", e4m3, i8)):
        for x, w in ((own, own), (u8, own), (own, u8), (u8, u8)):
            fn(**dict(make(), model=model(dtype), x=x(ROWS), W=w(N)))
        for x, w in ((other, own), (own, other)):
            with pytest.raises(B.TileShareError):
                fn(**dict(make(), model=model(dtype), x=x(ROWS), W=w(N)))
    fn, make = CALLS["norm_gate"]
    for dtype, own, other in (("int8", i8, e4m3), ("fp8", e4m3, i8)):
        fn(**dict(make(), model=model(dtype), xn=own(ROWS)))
        fn(**dict(make(), model=model(dtype), xn=u8(ROWS)))
        with pytest.raises(B.TileShareError):
            fn(**dict(make(), model=model(dtype), xn=other(ROWS)))
    fn(**dict(make(), model=model("bf16"), xn=z(ROWS, K, dtype=BF), xn_scale=None))
    for dtype in (torch.float16, torch.int16):
        refused(calls, "norm_gate", xn=z(ROWS, K, dtype=dtype), xn_scale=None)
    f32 = {n: z(ROWS, K) for n in ("x", "y", "x_out", "xn")}
    fn(**dict(make(), model=model("f32"), xn_scale=None, **f32))
    refused(calls, "norm_gate", **dict(f32, model=model("bf16"), xn_scale=None))
    refused(calls, "norm_gate", model=model("f32"), xn_scale=None, **dict(f32, y=z(ROWS, K, dtype=I32)))


def test_unknown_model_dtypes_are_refused(calls):
    refused(calls, "norm_gate", model=model(9))
    refused(calls, "linear_q8", model=model(9))
    refused(calls, "linear_q8", model=model("bf16"))


@pytest.mark.parametrize("name,tensor", [("quantize", "q"), ("linear", "y"), ("linear_q8", "y"), ("norm_gate", "y"),
                                         ("norm_gate", "x_out"), ("norm_gate", "xn")])
def test_rows_of_another_length_are_refused(calls, name, tensor):
    """Outputs are written row after row: one with longer rows, or with its sides exchanged, would be scrambled."""
    t = CALLS[name][1]()[tensor]
    rows, cols = t.shape
    for shape in ((rows, cols + 8), (2 * rows, cols // 2), (cols, rows), (rows, cols, 1)):
        refused(calls, name, **{tensor: torch.zeros(shape, dtype=t.dtype)})
    fn, make = CALLS[name]
    fn(**dict(make(), **{tensor: t.reshape(-1)}))                 # the same elements in one dimension
    fn(**dict(make(), **{tensor: t.reshape(2, rows // 2, cols)}))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("missing", ["y", "bias"])
def test_a_missing_tensor_of_a_linear_layer_is_an_error_of_the_call(calls, monkeypatch, dtype, missing):
    Bd.build()
    monkeypatch.setattr(B, "_lib", None)              # the library itself, which refuses it before anything runs
    args = CALLS["linear"][1]()
    args["model"] = B.model_desc(64, 4, 256, dtype, (0, 8, 8)) if dtype == "f32" else model(dtype)
    with pytest.raises(B.TileShareError) as e:
        B.op_linear(**dict(args, **{missing: None}))
    assert e.value.status == 1
