"""ctypes binding of libtileshare.so (include/tileshare.h, include/tileshare_ops.h).

Argument marshalling only: tensors are passed as device pointers with the current
CUDA stream, structs are filled field by field, and a non-zero status raises
TileShareError with the library's own message.  Every step of the computation
runs in the library's CUDA kernels.  The library must have been built
(``python -m shared_token_transformer_b200.build``); loading raises otherwise.
"""

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtileshare.so")

# ---------------------------------------------------------------------------
# C types
# ---------------------------------------------------------------------------
TS_OK = 0
TS_BLEND_LINEAR_RAMP = 0
TS_BLEND_HARD_STITCH = 1
TS_SHARE_QKV, TS_SHARE_OUT, TS_SHARE_MLP = 1, 2, 4
TS_F32, TS_BF16, TS_FP8_E4M3, TS_INT8 = 0, 1, 2, 3
TS_ROWS_SHARED, TS_ROWS_TILED = 0, 1
TS_EPI_BIAS, TS_EPI_BIAS_GELU, TS_EPI_BIAS_RESID, TS_EPI_BIAS_SWIGLU = 0, 1, 2, 3
TS_BLOCK_LN_GELU, TS_BLOCK_RMS_SWIGLU = 0, 1
BLOCKS = {"ln_gelu": TS_BLOCK_LN_GELU, "rms_swiglu": TS_BLOCK_RMS_SWIGLU}
DTYPES = {"f32": TS_F32, "bf16": TS_BF16, "fp8": TS_FP8_E4M3, "int8": TS_INT8}

_int3 = ctypes.c_int * 3
_cp = ctypes.c_void_p


class PlanDesc(ctypes.Structure):
    _fields_ = [("grid", _int3), ("win", _int3), ("stride", _int3),
                ("T", ctypes.c_int), ("U", ctypes.c_int), ("Nw", ctypes.c_int), ("N", ctypes.c_int),
                ("nnz", ctypes.c_int), ("max_cover", ctypes.c_int), ("device", ctypes.c_int),
                ("run", ctypes.c_int),
                ("origins", ctypes.POINTER(ctypes.c_int)), ("tile_tok", ctypes.POINTER(ctypes.c_int)),
                ("slot_pos", ctypes.POINTER(ctypes.c_int)), ("tok_ptr", ctypes.POINTER(ctypes.c_int)),
                ("tok_ent", ctypes.POINTER(ctypes.c_int)), ("wbar", ctypes.POINTER(ctypes.c_float)),
                ("R", ctypes.c_int)]


class ModelDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("heads", ctypes.c_int), ("mlp", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps_ln", ctypes.c_float), ("eps_qk", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("rope_dims", _int3), ("block", ctypes.c_int)]


_WEIGHT_FIELDS = ["ln1_g", "ln1_b", "w_qkv", "b_qkv", "q_g", "k_g", "w_o", "b_o", "ln2_g", "ln2_b",
                  "w_1", "b_1", "w_2", "b_2", "s_qkv", "s_o", "s_1", "s_2"]


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, _cp) for n in _WEIGHT_FIELDS]


class SandwichWeights(ctypes.Structure):
    _fields_ = [(n, _cp) for n in ("post1_g", "post1_b", "gate1", "scale1", "post2_g", "post2_b", "gate2", "scale2",
                                   "row_group")] + [("groups", ctypes.c_int)]


class NormGate(ctypes.Structure):
    _fields_ = [(n, _cp) for n in ("post_g", "post_b", "pre_g", "pre_b", "gate", "scale")] + \
        [("groups", ctypes.c_int)]


class TraceEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int), ("timed", ctypes.c_int),
                ("ms", ctypes.c_double), ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


class TileShareError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} -> status {status}: {msg}")
        self.status = status


# ---------------------------------------------------------------------------
# library loading
# ---------------------------------------------------------------------------
_lib = None

_SIGS = {
    "ts_plan_create": [ctypes.POINTER(ctypes.c_int)] * 3 + [ctypes.c_int, ctypes.POINTER(_cp)],
    "ts_plan_create_host": [ctypes.POINTER(ctypes.c_int)] * 3 + [ctypes.c_int, ctypes.POINTER(_cp)],
    "ts_plan_create_registers": [ctypes.POINTER(ctypes.c_int)] * 3 + [ctypes.c_int, ctypes.c_int, ctypes.POINTER(_cp)],
    "ts_plan_create_host_registers": [ctypes.POINTER(ctypes.c_int)] * 3 + [ctypes.c_int, ctypes.c_int,
                                                                            ctypes.POINTER(_cp)],
    "ts_plan_info": [_cp, ctypes.POINTER(PlanDesc)],
    "ts_plan_destroy": [_cp],
    "ts_workspace_size": [_cp, ctypes.POINTER(ModelDesc), ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "ts_block_tiled": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), _cp, _cp, ctypes.c_size_t, _cp],
    "ts_block_shared": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), _cp, _cp, ctypes.c_size_t, _cp],
    "ts_block_shared_noalloc": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), _cp, _cp],
    "ts_block_partial": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), ctypes.c_uint, _cp, _cp,
                         ctypes.c_size_t, _cp],
    "ts_decode_stack": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), ctypes.c_int, ctypes.c_int,
                        _cp, _cp, _cp, _cp, ctypes.c_size_t, _cp],
    "ts_quantize_rows_e4m3": [_cp, ctypes.c_int, ctypes.c_int, _cp, _cp, _cp],
    "ts_quantize_rows_i8": [_cp, ctypes.c_int, ctypes.c_int, _cp, _cp, _cp],
    "ts_gather_tiles": [_cp, ctypes.POINTER(ModelDesc), _cp, _cp, _cp, _cp],
    "ts_trace_begin": [ctypes.c_int],
    "ts_trace_end": [ctypes.POINTER(TraceEntry), ctypes.c_int, ctypes.POINTER(ctypes.c_int)],
    "ts_launch_count": [],
    "ts_device_status": [],
    "ts_selftest_bounded_wait": [ctypes.c_longlong, _cp, _cp],
    "ts_status_string": [ctypes.c_int],
    "ts_last_error": [],
    "ts_block_shared_sandwich": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights),
                                 ctypes.POINTER(SandwichWeights), _cp, _cp, ctypes.c_size_t, _cp],
    "ts_block_tiled_sandwich": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights),
                                ctypes.POINTER(SandwichWeights), _cp, _cp, ctypes.c_size_t, _cp],
    "ts_op_norm_gate": [_cp, ctypes.POINTER(NormGate), _cp, _cp, _cp, ctypes.c_int, _cp, _cp,
                        _cp, _cp],
    "ts_op_layernorm": [ctypes.POINTER(ModelDesc), _cp, ctypes.c_int, _cp, _cp, _cp, _cp],
    "ts_op_linear": [_cp, _cp, ctypes.c_int, ctypes.c_int, _cp, _cp, ctypes.c_int, _cp,
                     ctypes.c_int, _cp, _cp, _cp],
    "ts_op_linear_q8": [_cp, _cp, _cp, ctypes.c_int, ctypes.c_int, _cp, _cp, ctypes.c_int, _cp,
                        ctypes.c_int, _cp, _cp],
    "ts_op_qkv": [_cp, ctypes.POINTER(ModelDesc), ctypes.POINTER(LayerWeights), ctypes.c_int, _cp, _cp, _cp, _cp],
    "ts_op_attention": [_cp, ctypes.POINTER(ModelDesc), ctypes.c_int, _cp, _cp, _cp],
    "ts_op_merge": [_cp, ctypes.POINTER(ModelDesc), _cp, ctypes.c_int, _cp, _cp],
}


def lib():
    """Load libtileshare.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m shared_token_transformer_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = None if name == "ts_plan_destroy" else ctypes.c_int
        L.ts_launch_count.restype = ctypes.c_longlong
        L.ts_status_string.restype = ctypes.c_char_p
        L.ts_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(name, status):
    if status != TS_OK:
        raise TileShareError(name, status, lib().ts_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


_device = _raw_stream = None      # torch's current device number, and the stream of a device as an address
_f32 = _bf16 = _i32 = None        # torch's types
_rows_type = _q8_types = None     # by model dtype: the type of rows, and those that 8-bit rows may have (bytes, as the
                                  # quantisers fill them, or the type proper)


def _cuda():
    global _device, _raw_stream, _f32, _bf16, _i32, _rows_type, _q8_types
    import torch
    torch.cuda.init()
    _f32, _bf16, _i32 = torch.float32, torch.bfloat16, torch.int32
    _rows_type = {TS_F32: _f32, TS_BF16: _bf16, TS_FP8_E4M3: _bf16, TS_INT8: _bf16}
    _q8_types = {TS_F32: (), TS_BF16: (), TS_FP8_E4M3: (torch.float8_e4m3fn, torch.uint8), TS_INT8: (torch.int8, torch.uint8)}
    _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    return _device


def _stream(stream=None):
    """The cudaStream_t of `stream`, or of torch's current stream (as an address: torch's stream objects would take half
    the time of a call of a few microseconds)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        _cuda()
    return _raw_stream(_device())


def _unfit(fn):
    """quantize_rows_i8, op_linear of int8 models, op_linear_q8 and op_norm_gate take contiguous tensors of the current
    device whose types and sizes belong together; others are refused here, since a pointer does not tell."""
    raise TileShareError(fn, 1, "a tensor is not contiguous, of another type or shape, not on the current device, or too "
                                "small for the call")


def _holds(t, rows, cols):
    """Whether the contiguous t holds the rows one behind the other: [>= rows, cols], or flat."""
    return t.numel() >= rows * cols and t.dim() > 0 and (t.shape[-1] == cols or t.dim() == 1)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
class Plan:
    """ts_plan_t with its host arrays as NumPy views (copied)."""

    def __init__(self, grid, win, stride, host_only=False, rule=TS_BLEND_LINEAR_RAMP, registers=1):
        g, w, s = _int3(*grid), _int3(*win), _int3(*stride)
        h = _cp()
        fn = "ts_plan_create_host_registers" if host_only else "ts_plan_create_registers"
        _check(fn, getattr(lib(), fn)(g, w, s, rule, int(registers), ctypes.byref(h)))
        self.handle = h
        d = PlanDesc()
        _check("ts_plan_info", lib().ts_plan_info(h, ctypes.byref(d)))
        self.desc = d
        self.T, self.U, self.Nw, self.N, self.nnz = d.T, d.U, d.Nw, d.N, d.nnz
        self.max_cover, self.device, self.run, self.R = d.max_cover, d.device, d.run, d.R

        def arr(p, n, dt):
            return np.ctypeslib.as_array(p, shape=(n,)).astype(dt).copy()

        self.origins = arr(d.origins, 3 * d.T, np.int64).reshape(d.T, 3)
        self.tile_tok = arr(d.tile_tok, d.T * d.Nw, np.int64).reshape(d.T, d.Nw)
        self.slot_pos = arr(d.slot_pos, 3 * d.Nw, np.int64).reshape(d.Nw, 3)
        self.tok_ptr = arr(d.tok_ptr, d.U + 1, np.int64)
        self.tok_ent = arr(d.tok_ent, d.nnz, np.int64)
        self.wbar = arr(d.wbar, d.nnz, np.float32)

    def close(self):
        if self.handle is not None and self.handle.value:
            lib().ts_plan_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# model / weights
# ---------------------------------------------------------------------------
def model_desc(d, heads, mlp, dtype, rope_dims, eps_ln=1e-6, eps_qk=1e-6, rope_base=10000.0, block="ln_gelu"):
    return ModelDesc(d, heads, mlp, DTYPES[dtype] if isinstance(dtype, str) else dtype, eps_ln, eps_qk, rope_base,
                     _int3(*rope_dims), BLOCKS[block] if isinstance(block, str) else block)


def layer_weights(tensors):
    """ts_layer_weights from a dict of device tensors (missing names -> NULL).

    The struct keeps a reference to the tensors: their device memory stays
    allocated for as long as the struct is alive."""
    w = LayerWeights()
    for n in _WEIGHT_FIELDS:
        t = tensors.get(n)
        setattr(w, n, None if t is None else t.data_ptr())
    w._tensors = dict(tensors)
    return w


def _keep(struct, tensors):
    """Fill a struct of fp32 vectors [d], gates [groups, d] and an int32 row_group, and keep the tensors alive."""
    import torch
    width, groups, device = set(), set(), set()
    for n, t in tensors.items():
        if t is None:
            continue
        dtype = torch.int32 if n == "row_group" else torch.float32
        if not t.is_contiguous() or t.dtype is not dtype:
            raise ValueError(f"{n} must be contiguous and {dtype}")
        gate = n.startswith("gate")
        if n != "row_group" and (t.dim() == 0 or t.numel() == 0 or (t.numel() != t.shape[-1] and not gate)):
            raise ValueError(f"{n} must be [{'groups, ' if gate else ''}d], not {list(t.shape)}")
        setattr(struct, n, t.data_ptr())
        device.add(t.get_device())
        if gate:
            groups.add(t.numel() // t.shape[-1])     # a vector [d] is one group
        if n != "row_group":
            width.add(t.shape[-1])
    if len(groups) > 1 or len(width) > 1 or len(device) > 1:
        raise ValueError("the vectors have different widths or devices, or the gates different numbers of groups")
    struct.groups = groups.pop() if groups else 0
    struct.width = width.pop() if width else 0
    struct.device = device.pop() if device else None
    struct._tensors = dict(tensors)
    return struct


def norm_gate_desc(post_g=None, post_b=None, pre_g=None, pre_b=None, gate=None, scale=None):
    """ts_norm_gate of device tensors (fp32 [d]; gate [groups, d], or [d] for one group), kept alive by the struct."""
    return _keep(NormGate(), {"post_g": post_g, "post_b": post_b, "pre_g": pre_g, "pre_b": pre_b, "gate": gate,
                              "scale": scale})


def sandwich_weights(post1_g=None, post1_b=None, gate1=None, scale1=None, post2_g=None, post2_b=None, gate2=None,
                     scale2=None, row_group=None):
    """ts_sandwich_weights of device tensors (fp32, as norm_gate_desc, for both halves of a layer; row_group int32)."""
    return _keep(SandwichWeights(), {"post1_g": post1_g, "post1_b": post1_b, "gate1": gate1, "scale1": scale1,
                                     "post2_g": post2_g, "post2_b": post2_b, "gate2": gate2, "scale2": scale2,
                                     "row_group": row_group})


def workspace_size(plan, model, L=0, k=0):
    n = ctypes.c_size_t()
    _check("ts_workspace_size", lib().ts_workspace_size(plan.handle, ctypes.byref(model), L, k, ctypes.byref(n)))
    return n.value


# ---------------------------------------------------------------------------
# compute calls (device tensors, current stream)
# ---------------------------------------------------------------------------
def block_tiled(plan, model, weights, X, ws, stream=None):
    _check("ts_block_tiled", lib().ts_block_tiled(plan.handle, ctypes.byref(model), ctypes.byref(weights), _ptr(X),
                                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def block_shared(plan, model, weights, S, ws, stream=None):
    _check("ts_block_shared", lib().ts_block_shared(plan.handle, ctypes.byref(model), ctypes.byref(weights), _ptr(S),
                                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def block_partial(plan, model, weights, shared_ops, X, ws, stream=None):
    """ts_block_partial: per-tile states X, the TS_SHARE_* operations in shared_ops once per token."""
    _check("ts_block_partial", lib().ts_block_partial(plan.handle, ctypes.byref(model), ctypes.byref(weights),
                                                      int(shared_ops), _ptr(X), _ptr(ws),
                                                      ws.numel() * ws.element_size(), _stream(stream)))


def _sandwich_rows(fn, model, sandwich, rows):
    group = sandwich._tensors.get("row_group")
    if (sandwich.width not in (model.d, 0) or sandwich.device not in ((_device or _cuda())(), None) or
            (group is not None and group.numel() != rows)):
        raise TileShareError(fn, 1, f"sandwich vectors of another width or device, or a row_group not of {rows} rows")


def block_shared_sandwich(plan, model, weights, sandwich, S, ws, stream=None):
    """ts_block_shared_sandwich: block_shared with norms, gates and scales (sandwich_weights) around its halves."""
    _sandwich_rows("ts_block_shared_sandwich", model, sandwich, plan.U + plan.T * plan.R)
    _check("ts_block_shared_sandwich",
           lib().ts_block_shared_sandwich(plan.handle, ctypes.byref(model), ctypes.byref(weights),
                                          ctypes.byref(sandwich), _ptr(S), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)))


def block_tiled_sandwich(plan, model, weights, sandwich, X, ws, stream=None):
    """ts_block_tiled_sandwich: the same around block_tiled."""
    _sandwich_rows("ts_block_tiled_sandwich", model, sandwich, plan.T * plan.N)
    _check("ts_block_tiled_sandwich",
           lib().ts_block_tiled_sandwich(plan.handle, ctypes.byref(model), ctypes.byref(weights),
                                         ctypes.byref(sandwich), _ptr(X), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)))


def block_shared_noalloc(plan, model, weights, S, stream=None):
    """ts_block_shared with the library's static scratch instead of a workspace (allocates nothing)."""
    _check("ts_block_shared_noalloc", lib().ts_block_shared_noalloc(plan.handle, ctypes.byref(model),
                                                                    ctypes.byref(weights), _ptr(S), _stream(stream)))


def decode_stack(plan, model, weights_list, k, S0, G0, out, ws, stream=None):
    L = len(weights_list)
    arr = (LayerWeights * L)(*weights_list)      # copies of the structs; the originals keep the tensors alive
    _check("ts_decode_stack", lib().ts_decode_stack(plan.handle, ctypes.byref(model), arr, L, k, _ptr(S0), _ptr(G0),
                                                    _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                                    _stream(stream)))


def gather_tiles(plan, model, S0, G0, X, stream=None):
    _check("ts_gather_tiles", lib().ts_gather_tiles(plan.handle, ctypes.byref(model), _ptr(S0), _ptr(G0), _ptr(X),
                                                    _stream(stream)))


def trace_begin(max_launches=100000):
    _check("ts_trace_begin", lib().ts_trace_begin(max_launches))


def trace_end():
    """Per kernel class: dict name -> {launches, timed, ms, flops, bytes} (synchronises)."""
    cap = 64
    arr = (TraceEntry * cap)()
    n = ctypes.c_int()
    _check("ts_trace_end", lib().ts_trace_end(arr, cap, ctypes.byref(n)))
    return {arr[i].name.decode(): {"launches": arr[i].launches, "timed": arr[i].timed, "ms": arr[i].ms,
                                   "flops": arr[i].flops, "bytes": arr[i].bytes} for i in range(min(n.value, cap))}


def launch_count():
    return int(lib().ts_launch_count())


def quantize_rows_e4m3(x, q, scale, stream=None):
    rows, cols = x.shape
    _check("ts_quantize_rows_e4m3", lib().ts_quantize_rows_e4m3(_ptr(x), rows, cols, _ptr(q), _ptr(scale),
                                                                _stream(stream)))


def quantize_rows_i8(x, q, scale, stream=None):
    rows, cols = x.shape
    device = (_device or _cuda())()
    if not (x.dtype is _bf16 and q.dtype in _q8_types[TS_INT8] and scale.dtype is _f32 and
            (q.shape == x.shape or _holds(q, rows, cols)) and scale.nbytes >= 4 * rows and
            x.is_contiguous() and q.is_contiguous() and scale.is_contiguous() and
            x.get_device() == q.get_device() == scale.get_device() == device):
        _unfit("ts_quantize_rows_i8")
    _check("ts_quantize_rows_i8", lib().ts_quantize_rows_i8(_ptr(x), rows, cols, _ptr(q), _ptr(scale),
                                                            _stream(stream)))


def device_status():
    _check("ts_device_status", lib().ts_device_status())


def selftest_bounded_wait(limit_ns, done, stream=None):
    """ts_selftest_bounded_wait: a wait that nothing satisfies must time out (device int32 done[2])."""
    _check("ts_selftest_bounded_wait", lib().ts_selftest_bounded_wait(int(limit_ns), _ptr(done), _stream(stream)))


def op_layernorm(model, x, g, b, y, stream=None):
    _check("ts_op_layernorm", lib().ts_op_layernorm(ctypes.byref(model), _ptr(x), x.shape[0], _ptr(g), _ptr(b),
                                                    _ptr(y), _stream(stream)))


def op_norm_gate(model, gates, x, y, x_out, xn=None, xn_scale=None, row_group=None, stream=None):
    """ts_op_norm_gate: x_out = x + gate * scale * Norm_post(y) and xn = Norm_pre(x_out), as 8-bit rows with xn_scale."""
    shape = x.shape
    rows, d = shape
    device = (_device or _cuda())()
    dtype = model.dtype
    rows_type = _rows_type.get(dtype)
    if not (x.dtype is y.dtype is x_out.dtype is rows_type and d == model.d and (gates.width == d or gates.width == 0) and
            (gates.device == device or gates.device is None) and
            (shape == y.shape or (y.numel() == rows * d and _holds(y, rows, d))) and
            (shape == x_out.shape or _holds(x_out, rows, d)) and
            x.is_contiguous() and y.is_contiguous() and x_out.is_contiguous() and
            x.get_device() == y.get_device() == x_out.get_device() == device):
        _unfit("ts_op_norm_gate")
    if xn is not None and not (
            xn.is_contiguous() and xn.get_device() == device and (shape == xn.shape or _holds(xn, rows, d)) and
            (xn.dtype is rows_type if xn_scale is None else
             xn.dtype in _q8_types[dtype] and xn_scale.dtype is _f32 and xn_scale.is_contiguous() and
             xn_scale.nbytes >= 4 * rows and xn_scale.get_device() == device)):
        _unfit("ts_op_norm_gate")
    if row_group is not None and not (row_group.dtype is _i32 and row_group.is_contiguous() and
                                      row_group.numel() == rows and row_group.get_device() == device):
        _unfit("ts_op_norm_gate")
    status = (_lib or lib()).ts_op_norm_gate(
        ctypes.addressof(model), gates, x.data_ptr(), y.data_ptr(),
        None if row_group is None else row_group.data_ptr(), rows, x_out.data_ptr(),
        None if xn is None else xn.data_ptr(), None if xn_scale is None else xn_scale.data_ptr(),
        _raw_stream(device) if stream is None else stream.cuda_stream)
    if status:
        _check("ts_op_norm_gate", status)


def op_linear(model, x, W, bias, y, epi=TS_EPI_BIAS, w_scale=None, scratch=None, stream=None):
    rows, K = x.shape
    wide = W.shape[0]
    N = wide // 2 if epi == TS_EPI_BIAS_SWIGLU else wide     # output width
    if model.dtype == TS_INT8:
        device = (_device or _cuda())()
        if not (bias is not None and y is not None and w_scale is not None and scratch is not None and
                x.dtype is y.dtype is _bf16 and W.dtype in _q8_types[TS_INT8] and bias.dtype is w_scale.dtype is _f32 and W.nbytes == wide * K and
                (y.shape == (rows, N) or _holds(y, rows, N)) and bias.nbytes >= 4 * wide <= w_scale.nbytes and
                scratch.nbytes >= rows * (K + 4) and x.is_contiguous() and W.is_contiguous() and y.is_contiguous() and
                bias.is_contiguous() and w_scale.is_contiguous() and scratch.is_contiguous() and
                x.get_device() == y.get_device() == W.get_device() == bias.get_device() == w_scale.get_device() ==
                scratch.get_device() == device):
            _unfit("ts_op_linear")
        st = _raw_stream(device) if stream is None else stream.cuda_stream
    else:
        st = _stream(stream)
    status = (_lib or lib()).ts_op_linear(ctypes.addressof(model), x.data_ptr(), rows, K, W.data_ptr(),
                                          None if w_scale is None else w_scale.data_ptr(), N,
                                          None if bias is None else bias.data_ptr(), epi,
                                          None if y is None else y.data_ptr(),
                                          None if scratch is None else scratch.data_ptr(), st)
    if status:
        _check("ts_op_linear", status)


def op_linear_q8(model, x, x_scale, W, w_scale, bias, y, epi=TS_EPI_BIAS, stream=None):
    """ts_op_linear_q8: the linear layer of rows that are 8-bit already, with their scales."""
    rows, K = x.shape
    wide = W.shape[0]
    N = wide // 2 if epi == TS_EPI_BIAS_SWIGLU else wide     # output width
    device = (_device or _cuda())()
    q8 = _q8_types.get(model.dtype, ())
    if not (x.dtype in q8 and W.dtype in q8 and y.dtype is _bf16 and x_scale.dtype is w_scale.dtype is bias.dtype is _f32 and
            W.nbytes == wide * K and (y.shape == (rows, N) or _holds(y, rows, N)) and
            bias.nbytes >= 4 * wide <= w_scale.nbytes and x_scale.nbytes >= 4 * rows and x.is_contiguous() and
            W.is_contiguous() and y.is_contiguous() and bias.is_contiguous() and w_scale.is_contiguous() and
            x_scale.is_contiguous() and
            x.get_device() == y.get_device() == W.get_device() == bias.get_device() == w_scale.get_device() ==
            x_scale.get_device() == device):
        _unfit("ts_op_linear_q8")
    status = (_lib or lib()).ts_op_linear_q8(ctypes.addressof(model), x.data_ptr(), x_scale.data_ptr(), rows, K,
                                             W.data_ptr(), w_scale.data_ptr(), N, bias.data_ptr(), epi, y.data_ptr(),
                                             _raw_stream(device) if stream is None else stream.cuda_stream)
    if status:
        _check("ts_op_linear_q8", status)


def op_qkv(plan, model, weights, mode, state, qkv, scratch, stream=None):
    _check("ts_op_qkv", lib().ts_op_qkv(plan.handle, ctypes.byref(model), ctypes.byref(weights), mode, _ptr(state),
                                        _ptr(qkv), _ptr(scratch), _stream(stream)))


def op_attention(plan, model, mode, qkv, O, stream=None):
    _check("ts_op_attention", lib().ts_op_attention(plan.handle, ctypes.byref(model), mode, _ptr(qkv), _ptr(O),
                                                    _stream(stream)))


def op_merge(plan, model, P, rows, A, stream=None):
    _check("ts_op_merge", lib().ts_op_merge(plan.handle, ctypes.byref(model), _ptr(P), rows, _ptr(A),
                                            _stream(stream)))
