"""Python binding of the MI355X probabilistic-circuit sum-layer library.

Thin ctypes marshalling over the C ABI declared in ``include/pc.h``: the
functions here carry the C names, check argument types and sizes, and pass
device pointers of torch tensors and the current HIP stream.  Every step of
the computation runs in the library's HIP kernels; there is no fallback.  The
library is ``libpc.so`` next to this file, built by ``log_space_sum_amd.build``.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpc.so")

PC_OK, PC_ERR_INVALID_ARG, PC_ERR_UNSUPPORTED, PC_ERR_WORKSPACE, PC_ERR_HIP, PC_ERR_NO_DEVICE = range(6)
PC_PREC_AUTO, PC_PREC_FP32, PC_PREC_TF32 = 0, 1, 2
PC_LAYER_INPUT_CAT, PC_LAYER_INPUT_EXTERNAL, PC_LAYER_PRODUCT, PC_LAYER_SUM = 0, 1, 2, 3
PC_CLASS_SHARED, PC_CLASS_STRIDED, PC_CLASS_GENERAL, PC_CLASS_LOWRANK = 0, 1, 2, 3
PC_BWD_SEEDED = 1
PC_LOWRANK_EXP_SUM, PC_LOWRANK_SUM_EXP = 0, 1
LOWRANK_FORMS = {"exp_sum": PC_LOWRANK_EXP_SUM, "sum_exp": PC_LOWRANK_SUM_EXP}
PC_NUM_KERNEL_KINDS = 16
KERNEL_KINDS = ["sum_fwd_gemm", "elem_flow_gemm", "param_flow_gemm", "weight_split", "column_max",
                "exp_children", "scaled_flows", "input_fwd", "input_bwd", "product_fwd",
                "product_bwd", "em", "lowrank_fwd", "lowrank_bwd", "other", "lowrank_coef"]
MODES = {"auto": PC_PREC_AUTO, "fp32": PC_PREC_FP32, "tf32": PC_PREC_TF32}
GEMM_KINDS = {"fwd": 0, "elem": 1, "param": 2}

PC_DTYPE_F32, PC_DTYPE_BF16, PC_DTYPE_F16 = range(3)

_i32p = C.POINTER(C.c_int32)


class pc_sum_group(C.Structure):
    _fields_ = [("out_start", C.c_int32), ("num_nodes", C.c_int32), ("num_ch_blocks", C.c_int32),
                ("ch_block_size", C.c_int32), ("ch_block_start", _i32p), ("param_offset", C.c_int64),
                ("lowrank_slot", C.c_int32)]


class pc_layer_desc(C.Structure):
    _fields_ = [("kind", C.c_int32), ("node_start", C.c_int32), ("num_nodes", C.c_int32),
                ("num_cats", C.c_int32), ("num_rows", C.c_int32), ("param_offset", C.c_int64),
                ("var", _i32p), ("row", _i32p), ("ch_ptr", _i32p), ("ch_ids", _i32p),
                ("num_groups", C.c_int32), ("groups", C.POINTER(pc_sum_group))]


class pc_circuit_desc(C.Structure):
    _fields_ = [("num_nodes", C.c_int32), ("num_vars", C.c_int32), ("num_params", C.c_int64),
                ("num_layers", C.c_int32), ("layers", C.POINTER(pc_layer_desc)), ("root", C.c_int32),
                ("lowrank_rank", C.c_int32), ("lowrank_form", C.c_int32)]


class pc_lowrank_io(C.Structure):
    _fields_ = [("num_slots", C.c_int32), ("A", C.POINTER(C.c_void_p)), ("B", C.POINTER(C.c_void_p)),
                ("dA", C.POINTER(C.c_void_p)), ("dB", C.POINTER(C.c_void_p)), ("z_flows", C.c_void_p)]


class pc_layout_summary(C.Structure):
    _fields_ = [("num_layers", C.c_int32), ("num_sum_layers", C.c_int32), ("num_param_blocks", C.c_int32),
                ("num_row_segments", C.c_int32), ("num_params", C.c_int64), ("num_outputs", C.c_int32),
                ("device", C.c_int32)]


class pc_heads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class pc_linear_attention(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("heads", C.c_int32), ("kv_heads", C.c_int32), ("dim_k", C.c_int32),
                ("dim_v", C.c_int32), ("num_seqs", C.c_int32), ("num_tokens", C.c_int64), ("max_seqlen", C.c_int64),
                ("cu_seqlens", C.c_void_p), ("log_decay", C.c_void_p), ("scale", C.c_float),
                ("q", pc_heads), ("k", pc_heads), ("v", pc_heads), ("o", pc_heads),
                ("state_in", C.c_void_p), ("state_out", C.c_void_p),
                ("d_o", pc_heads), ("d_q", pc_heads), ("d_k", pc_heads), ("d_v", pc_heads),
                ("dstate_out", C.c_void_p), ("dstate_in", C.c_void_p),
                ("state", C.c_void_p), ("num_slots", C.c_int64), ("slots", C.c_void_p)]


class pc_pages(C.Structure):
    _fields_ = [("data", C.c_void_p), ("page_stride", C.c_int64), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class pc_attention(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("heads", C.c_int32), ("kv_heads", C.c_int32), ("dim_k", C.c_int32),
                ("dim_v", C.c_int32), ("num_seqs", C.c_int32), ("num_tokens", C.c_int64), ("cu_seqlens", C.c_void_p),
                ("scale", C.c_float), ("q", pc_heads), ("k", pc_heads), ("v", pc_heads), ("o", pc_heads),
                ("lse", C.c_void_p), ("d_o", pc_heads), ("d_q", pc_heads), ("d_k", pc_heads), ("d_v", pc_heads),
                ("k_cache", pc_pages), ("v_cache", pc_pages), ("num_pages", C.c_int32), ("page_size", C.c_int32),
                ("max_pages", C.c_int32), ("page_table", C.c_void_p), ("page_table_stride", C.c_int64),
                ("cached", C.c_void_p), ("max_seqlen", C.c_int64), ("max_length", C.c_int64)]


class pc_rotary(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("heads", C.c_int32), ("kv_heads", C.c_int32), ("dim", C.c_int32),
                ("num_tokens", C.c_int64), ("rotary_dim", C.c_int32), ("interleaved", C.c_int32), ("norm", C.c_int32),
                ("eps", C.c_float), ("magnitude", C.c_float), ("positions", C.c_void_p), ("freq", C.c_void_p),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("q", pc_heads), ("k", pc_heads),
                ("q_out", pc_heads), ("k_out", pc_heads), ("d_q_out", pc_heads), ("d_k_out", pc_heads),
                ("d_q", pc_heads), ("d_k", pc_heads), ("d_q_weight", C.c_void_p), ("d_k_weight", C.c_void_p)]


ROTARY_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}

EXPORTS = {
    "pc_compile_layout": (C.c_int, [C.POINTER(pc_circuit_desc), C.c_int, C.POINTER(C.c_void_p)]),
    "pc_destroy": (C.c_int, [C.c_void_p]),
    "pc_set_precision": (C.c_int, [C.c_void_p, C.c_int]),
    "pc_get_precision": (C.c_int, [C.c_void_p, C.POINTER(C.c_int)]),
    "pc_set_split": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int]),
    "pc_set_option": (C.c_int, [C.c_void_p, C.c_int, C.c_int]),
    "pc_workspace_bytes": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_size_t)]),
    "pc_forward": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                             C.POINTER(pc_lowrank_io), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_forward_static": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                    C.POINTER(pc_lowrank_io), C.c_void_p]),
    "pc_backward": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_int, C.POINTER(pc_lowrank_io), C.c_void_p, C.c_size_t,
                              C.c_void_p]),
    "pc_em_step": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_float, C.c_float, C.c_void_p]),
    "pc_em_step_corrected": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_float, C.c_float,
                                       C.c_void_p]),
    "pc_layer_norm_forward": (C.c_int, [C.c_int, C.c_int, C.c_int64, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p,
                                        C.c_void_p, C.c_float, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                        C.c_void_p]),
    "pc_layer_norm_workspace_bytes": (C.c_int, [C.c_int64, C.c_int32, C.POINTER(C.c_size_t)]),
    "pc_layer_norm_backward": (C.c_int, [C.c_int, C.c_int, C.c_int64, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p,
                                         C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64,
                                         C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_linear_attention_workspace_bytes": (C.c_int, [C.POINTER(pc_linear_attention), C.c_int, C.POINTER(C.c_size_t)]),
    "pc_linear_attention_forward": (C.c_int, [C.c_int, C.POINTER(pc_linear_attention), C.c_void_p, C.c_size_t,
                                              C.c_void_p]),
    "pc_linear_attention_backward": (C.c_int, [C.c_int, C.POINTER(pc_linear_attention), C.c_void_p, C.c_size_t,
                                               C.c_void_p]),
    "pc_linear_attention_step": (C.c_int, [C.c_int, C.POINTER(pc_linear_attention), C.c_void_p]),
    "pc_orthogonalize_workspace_bytes": (C.c_int, [C.c_int, C.c_int64, C.c_int32, C.c_int32, C.POINTER(C.c_size_t)]),
    "pc_orthogonalize": (C.c_int, [C.c_int, C.c_int, C.c_int64, C.c_int32, C.c_int32, C.c_void_p, C.c_int64, C.c_int64,
                                   C.c_void_p, C.c_int64, C.c_int64, C.c_int32, C.POINTER(C.c_float), C.c_float,
                                   C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_rotary_frequencies": (C.c_int, [C.c_int32, C.c_double, C.c_int, C.c_double, C.c_double, C.c_double, C.c_double,
                                        C.POINTER(C.c_double)]),
    "pc_rotary_forward": (C.c_int, [C.c_int, C.POINTER(pc_rotary), C.c_void_p]),
    "pc_rotary_workspace_bytes": (C.c_int, [C.POINTER(pc_rotary), C.POINTER(C.c_size_t)]),
    "pc_rotary_backward": (C.c_int, [C.c_int, C.POINTER(pc_rotary), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_attention_workspace_bytes": (C.c_int, [C.POINTER(pc_attention), C.c_int, C.POINTER(C.c_size_t)]),
    "pc_attention_forward": (C.c_int, [C.c_int, C.POINTER(pc_attention), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_attention_backward": (C.c_int, [C.c_int, C.POINTER(pc_attention), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_attention_cached_workspace_bytes": (C.c_int, [C.POINTER(pc_attention), C.POINTER(C.c_size_t)]),
    "pc_attention_cached": (C.c_int, [C.c_int, C.POINTER(pc_attention), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pc_last_error": (C.c_char_p, []),
    "pc_layout_info": (C.c_int, [C.c_void_p, C.POINTER(pc_layout_summary)]),
    "pc_layer_class": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_int)]),
    "pc_set_timing": (C.c_int, [C.c_void_p, C.c_int]),
    "pc_kernel_times": (C.c_int, [C.c_void_p, C.POINTER(C.c_int64), C.POINTER(C.c_double)]),
}

_lib = None


class PCError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"[pc error {code}] {msg}")
        self.code = code


def load_library(path: str):
    """A build of the library at `path`, its calls typed (does not make it
    the one the binding uses; see using_library)."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m log_space_sum_amd.build`")
    L = C.CDLL(path)
    for name, (res, args) in EXPORTS.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def lib():
    """The loaded libpc.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load_library(LIB_PATH)
    return _lib


class using_library:
    """Context in which the binding's calls go to another build of the
    library (loaded with load_library; handles compiled meanwhile keep it)."""

    def __init__(self, path: str):
        self.other = load_library(path)

    def __enter__(self):
        global _lib
        self.saved = lib()
        _lib = self.other
        return self.other

    def __exit__(self, *exc):
        global _lib
        _lib = self.saved
        return False


def _check(code):
    if code != PC_OK:
        raise PCError(code, lib().pc_last_error().decode())


def pc_last_error() -> str:
    return lib().pc_last_error().decode()


# ---------------------------------------------------------------------------
# descriptor marshalling
# ---------------------------------------------------------------------------

def _i32(a):
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return arr, arr.ctypes.data_as(_i32p)


class Handle:
    """Owns a pc_handle (destroyed with the object)."""

    def __init__(self, ptr, circuit):
        self.ptr = ptr
        self.lib = lib()             # the build that made it frees it
        self.num_nodes = circuit.num_nodes
        self.num_params = circuit.num_params
        self.num_vars = circuit.num_vars
        self.root = circuit.root

    def __del__(self):
        if getattr(self, "ptr", None) and getattr(self, "lib", None) is not None:
            self.lib.pc_destroy(self.ptr)
            self.ptr = None


def pc_compile_layout(circuit, device: int = 0) -> Handle:
    """Compile a circuit (an object with num_nodes, num_vars, num_params, root,
    lowrank_rank and a list of layers with the fields of pc_layer_desc /
    pc_sum_group) into a handle; device < 0 compiles host-only."""
    keep = []
    layers = (pc_layer_desc * len(circuit.layers))()
    for i, ly in enumerate(circuit.layers):
        d = layers[i]
        if hasattr(ly, "groups"):
            d.kind = PC_LAYER_SUM
            gs = (pc_sum_group * len(ly.groups))()
            for k, g in enumerate(ly.groups):
                arr, p = _i32(g.ch_block_start)
                keep.append(arr)
                gs[k].out_start = int(g.out_start)
                gs[k].num_nodes = int(g.num_nodes)
                gs[k].num_ch_blocks = int(len(arr))
                gs[k].ch_block_size = int(g.ch_block_size)
                gs[k].ch_block_start = p
                gs[k].param_offset = int(g.param_offset)
                gs[k].lowrank_slot = int(getattr(g, "lowrank", -1))
            keep.append(gs)
            d.num_groups = len(ly.groups)
            d.groups = gs
        elif hasattr(ly, "ch_ptr"):
            d.kind = PC_LAYER_PRODUCT
            d.node_start, d.num_nodes = int(ly.node_start), int(ly.num_nodes)
            a1, d.ch_ptr = _i32(ly.ch_ptr)
            a2, d.ch_ids = _i32(ly.ch_ids)
            keep += [a1, a2]
        elif hasattr(ly, "num_cats"):
            d.kind = PC_LAYER_INPUT_CAT
            d.node_start, d.num_nodes = int(ly.node_start), int(ly.num_nodes)
            d.num_cats, d.num_rows = int(ly.num_cats), int(ly.num_rows)
            d.param_offset = int(ly.param_offset)
            a1, d.var = _i32(ly.var)
            a2, d.row = _i32(ly.row)
            keep += [a1, a2]
        else:
            d.kind = PC_LAYER_INPUT_EXTERNAL
            d.node_start, d.num_nodes = int(ly.node_start), int(ly.num_nodes)
    desc = pc_circuit_desc(num_nodes=int(circuit.num_nodes), num_vars=int(circuit.num_vars),
                           num_params=int(circuit.num_params), num_layers=len(circuit.layers),
                           layers=layers, root=int(circuit.root),
                           lowrank_rank=int(getattr(circuit, "lowrank_rank", 0)),
                           lowrank_form=LOWRANK_FORMS[getattr(circuit, "lowrank_form", "exp_sum")])
    out = C.c_void_p()
    _check(lib().pc_compile_layout(C.byref(desc), int(device), C.byref(out)))
    return Handle(out, circuit)


def pc_destroy(h: Handle):
    if h.ptr:
        _check(lib().pc_destroy(h.ptr))
        h.ptr = None


def pc_set_precision(h: Handle, mode):
    _check(lib().pc_set_precision(h.ptr, MODES.get(mode, mode) if isinstance(mode, str) else int(mode)))


def pc_get_precision(h: Handle) -> int:
    m = C.c_int()
    _check(lib().pc_get_precision(h.ptr, C.byref(m)))
    return m.value


def pc_set_split(h: Handle, mode, gemm_kind, planes_a: int, planes_b: int):
    mode = MODES.get(mode, mode) if isinstance(mode, str) else mode
    gemm_kind = GEMM_KINDS.get(gemm_kind, gemm_kind) if isinstance(gemm_kind, str) else gemm_kind
    _check(lib().pc_set_split(h.ptr, int(mode), int(gemm_kind), int(planes_a), int(planes_b)))


OPTIONS = {"layer_tile": 0, "param_tile": 1, "split_max": 2, "fuse": 3, "param_chunk": 4, "lr_pack": 5,
           "sumexp_fused": 6, "flow_fp8": 7}


def pc_set_option(h: Handle, option, value: int):
    """Kernel tuning: layer_tile (0 auto, 1 128x128, 2 256x128, 3 128x256, 4 128x64, 5 64x128), param_tile
    (0 auto, 1 128x128, 2 256x256, 3 128x256), split_max (1, 2, 4, 8), fuse (1: product
    layers inside the adjacent sum layer's kernels, 0: separate launches),
    param_chunk (-1 automatic; 0: parameter flows in one product at the end;
    n: in chunks of n tied copies on a second stream, overlapping the element
    flows), sumexp_fused (1: LowRank "sum_exp" through the fused kernels),
    flow_fp8 (1: the "sum_exp" parameter flows and denominator statistic from
    e4m3 operands in auto mode)."""
    option = OPTIONS.get(option, option) if isinstance(option, str) else option
    _check(lib().pc_set_option(h.ptr, int(option), int(value)))


def pc_workspace_bytes(h: Handle, batch: int) -> int:
    n = C.c_size_t()
    _check(lib().pc_workspace_bytes(h.ptr, int(batch), C.byref(n)))
    return n.value


def pc_layout_info(h: Handle) -> dict:
    s = pc_layout_summary()
    _check(lib().pc_layout_info(h.ptr, C.byref(s)))
    return {f: getattr(s, f) for f, _ in pc_layout_summary._fields_}


def pc_layer_class(h: Handle, layer: int) -> int:
    c = C.c_int()
    _check(lib().pc_layer_class(h.ptr, int(layer), C.byref(c)))
    return c.value


def pc_set_timing(h: Handle, enable: bool):
    _check(lib().pc_set_timing(h.ptr, 1 if enable else 0))


def pc_kernel_times(h: Handle) -> dict:
    n = (C.c_int64 * PC_NUM_KERNEL_KINDS)()
    ms = (C.c_double * PC_NUM_KERNEL_KINDS)()
    _check(lib().pc_kernel_times(h.ptr, n, ms))
    return {KERNEL_KINDS[k]: (int(n[k]), float(ms[k])) for k in range(PC_NUM_KERNEL_KINDS)}


# ---------------------------------------------------------------------------
# passes (torch tensors: device memory and streams only)
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t, dtype, numel=None, what="tensor"):
    if t is None:
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must live on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{what} has {t.numel()} elements, needs {numel}")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return C.c_void_p(int(stream))
    return C.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _lowrank_io(lowrank, grads=None, z_flows=None, num_params=None):
    """lowrank: list of (A, B) device tensors per slot; grads: list of (dA, dB);
    z_flows: the LowRank denominator statistic's accumulator ([num_params])."""
    if lowrank is None:
        return None, None
    torch = _torch()
    n = len(lowrank)
    A = (C.c_void_p * n)(*[_ptr(a, torch.float32, what="A").value for a, _ in lowrank])
    Bf = (C.c_void_p * n)(*[_ptr(b, torch.float32, what="B").value for _, b in lowrank])
    if grads is not None:
        dA = (C.c_void_p * n)(*[_ptr(a, torch.float32, what="dA").value for a, _ in grads])
        dB = (C.c_void_p * n)(*[_ptr(b, torch.float32, what="dB").value for _, b in grads])
    else:
        dA = dB = None
    z = _ptr(z_flows, torch.float32, num_params, "z_flows") if z_flows is not None else None
    io = pc_lowrank_io(num_slots=n, A=A, B=Bf, dA=dA, dB=dB, z_flows=z)
    return io, (A, Bf, dA, dB)


def pc_forward(h: Handle, batch: int, tokens, params, node_vals, ll=None, lowrank=None, ws=None,
               stream=None):
    torch = _torch()
    io, keep = _lowrank_io(lowrank)
    need = pc_workspace_bytes(h, batch)
    _check(lib().pc_forward(
        h.ptr, int(batch), _ptr(tokens, torch.int32, batch * h.num_vars, "tokens"),
        _ptr(params, torch.float32, h.num_params, "params"),
        _ptr(node_vals, torch.float32, h.num_nodes * batch, "node_vals"),
        _ptr(ll, torch.float32, batch, "ll"), C.byref(io) if io is not None else None,
        _ptr(ws, torch.uint8, need, "ws"), C.c_size_t(ws.numel() if ws is not None else 0),
        _stream(stream)))


def pc_forward_static(h: Handle, batch: int, tokens, params, node_vals, ll=None, lowrank=None, stream=None):
    """pc_forward without a workspace: the library's static device scratch
    (forward only; calls overlapping on one device race)."""
    torch = _torch()
    io, keep = _lowrank_io(lowrank)
    _check(lib().pc_forward_static(
        h.ptr, int(batch), _ptr(tokens, torch.int32, batch * h.num_vars, "tokens"),
        _ptr(params, torch.float32, h.num_params, "params"),
        _ptr(node_vals, torch.float32, h.num_nodes * batch, "node_vals"),
        _ptr(ll, torch.float32, batch, "ll"), C.byref(io) if io is not None else None, _stream(stream)))


def pc_backward(h: Handle, batch: int, tokens, params, node_vals, node_flows, param_flows, flags=0,
                lowrank=None, grads=None, ws=None, stream=None, z_flows=None):
    torch = _torch()
    io, keep = _lowrank_io(lowrank, grads, z_flows, h.num_params)
    need = pc_workspace_bytes(h, batch)
    _check(lib().pc_backward(
        h.ptr, int(batch), _ptr(tokens, torch.int32, batch * h.num_vars, "tokens"),
        _ptr(params, torch.float32, h.num_params, "params"),
        _ptr(node_vals, torch.float32, h.num_nodes * batch, "node_vals"),
        _ptr(node_flows, torch.float32, h.num_nodes * batch, "node_flows"),
        _ptr(param_flows, torch.float32, h.num_params, "param_flows"), int(flags),
        C.byref(io) if io is not None else None,
        _ptr(ws, torch.uint8, need, "ws"), C.c_size_t(ws.numel() if ws is not None else 0),
        _stream(stream)))


def pc_em_step(h: Handle, params, param_flows, step_size=1.0, pseudocount=0.0, stream=None):
    torch = _torch()
    _check(lib().pc_em_step(h.ptr, _ptr(params, torch.float32, h.num_params, "params"),
                            _ptr(param_flows, torch.float32, h.num_params, "param_flows"),
                            C.c_float(step_size), C.c_float(pseudocount), _stream(stream)))


def pc_em_step_corrected(h: Handle, params, param_flows, z_flows, step_size=1.0, pseudocount=0.0, stream=None):
    torch = _torch()
    _check(lib().pc_em_step_corrected(h.ptr, _ptr(params, torch.float32, h.num_params, "params"),
                                      _ptr(param_flows, torch.float32, h.num_params, "param_flows"),
                                      _ptr(z_flows, torch.float32, h.num_params, "z_flows"),
                                      C.c_float(step_size), C.c_float(pseudocount), _stream(stream)))


def workspace(h: Handle, batch: int, device="cuda", all_modes=False):
    """A workspace tensor (uint8) of pc_workspace_bytes(h, batch) bytes; with
    all_modes, the largest over both precision modes (so the handle's mode
    can change while the workspace stays)."""
    n = pc_workspace_bytes(h, batch)
    if all_modes:
        mode = pc_get_precision(h)
        for m in (PC_PREC_AUTO, PC_PREC_FP32):
            pc_set_precision(h, m)
            n = max(n, pc_workspace_bytes(h, batch))
        pc_set_precision(h, mode)
    return _torch().empty(max(n, 1), dtype=_torch().uint8, device=device)


# ---------------------------------------------------------------------------
# operators of the network in front of a conditional circuit (no handle)
# ---------------------------------------------------------------------------

# (These calls can be a few microseconds of device work, so their checks are
# kept to a few attribute reads; what is wrong is found out when something is.)

_DTYPES = None


def _dtype(t, what):
    global _DTYPES
    if _DTYPES is None:
        torch = _torch()
        _DTYPES = {torch.float32: PC_DTYPE_F32, torch.bfloat16: PC_DTYPE_BF16, torch.float16: PC_DTYPE_F16}
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _device(t, what):
    """The index of the GPU that the tensor lives on."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must live on the GPU")
    return dev


def _wrong(t, dev, dtype, shape, what):
    if _device(t, what) != dev:
        raise ValueError(f"{what} is on {t.device}, not on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _operand(t, dev, dtype, shape, what):
    """The data pointer of a tensor of this device, dtype and shape whose last
    dimension has stride 1 (any other strides)."""
    try:
        ok = t.get_device() == dev and t.dtype == dtype and t.shape == shape
    except AttributeError:
        ok = False
    if not ok:
        _wrong(t, dev, dtype, shape, what)
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"the last dimension of {what} must have stride 1")
    return t.data_ptr()


def _dense(t, dev, dtype, shape, what):
    """_operand of a contiguous tensor; None stays None."""
    if t is None:
        return None
    p = _operand(t, dev, dtype, shape, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return p


def _ws_ptr(ws, dev):
    """(pointer, bytes) of a workspace (the library checks its size)."""
    if ws is None:
        return None, 0
    n = ws.numel()
    return _dense(ws, dev, _torch().uint8, (n,), "ws"), n


def _stream_of(dev, stream):
    """The given stream, else the current one of the device."""
    if stream is not None:
        return int(stream)
    return _raw_stream(dev)


def _raw_stream(dev):
    global _raw_stream
    torch = _torch()     # the handle itself where torch hands it out, without an object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(dev)


def _bytes(f, *args):
    n = C.c_size_t()
    _check(f(*args, C.byref(n)))
    return n.value


def _matrix(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    return t


def pc_layer_norm_forward(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = layer norm of the rows of x [rows, cols] (rows may be strided); weight, bias: float32 [cols] or None;
    mean, rstd: float32 [rows], kept for the backward pass, or None."""
    dev, f32 = _device(_matrix(x, "x"), "x"), _torch().float32
    shape, dt = x.shape, x.dtype
    rows, cols = shape
    px, py = _operand(x, dev, dt, shape, "x"), _operand(y, dev, dt, shape, "y")
    _check(lib().pc_layer_norm_forward(
        dev, _dtype(x, "x"), rows, cols, px, x.stride(0), _dense(weight, dev, f32, (cols,), "weight"),
        _dense(bias, dev, f32, (cols,), "bias"), eps, py, y.stride(0), _dense(mean, dev, f32, (rows,), "mean"),
        _dense(rstd, dev, f32, (rows,), "rstd"), _stream_of(dev, stream)))


def layer_norm_workspace(rows: int, cols: int, device="cuda"):
    """A workspace tensor for pc_layer_norm_backward."""
    n = _bytes(lib().pc_layer_norm_workspace_bytes, int(rows), int(cols))
    return _torch().empty(n, dtype=_torch().uint8, device=device)


def pc_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, ws=None, stream=None):
    """dx, dweight and dbias (float32 [cols], or None; all overwritten) from dy, x and the forward's mean and rstd;
    ws: layer_norm_workspace(rows, cols), needed for dweight and dbias."""
    dev, f32 = _device(_matrix(x, "x"), "x"), _torch().float32
    shape, dt = x.shape, x.dtype
    rows, cols = shape
    px = _operand(x, dev, dt, shape, "x")
    pdy, pdx = _operand(dy, dev, dt, shape, "dy"), _operand(dx, dev, dt, shape, "dx")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_layer_norm_backward(
        dev, _dtype(x, "x"), rows, cols, pdy, dy.stride(0), px, x.stride(0), _dense(weight, dev, f32, (cols,), "weight"),
        _dense(mean, dev, f32, (rows,), "mean"), _dense(rstd, dev, f32, (rows,), "rstd"), pdx, dx.stride(0),
        _dense(dweight, dev, f32, (cols,), "dweight"), _dense(dbias, dev, f32, (cols,), "dbias"), pws, nws,
        _stream_of(dev, stream)))


def _heads(to, t, dev, dtype, shape, what):
    to.data = _operand(t, dev, dtype, shape, what)
    to.token_stride, to.head_stride, _ = t.stride()


def _attention(q, k, v, log_decay, scale):
    """The descriptor of q [tokens, heads, dim_k], k [tokens, kv_heads, dim_k], v [tokens, kv_heads, dim_v]."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must have three dimensions (tokens, heads, dim)")
    dev, dt = _device(q, "q"), q.dtype
    T, H, dk = q.shape
    K, dv = k.shape[1], v.shape[2]
    d = pc_linear_attention(_dtype(q, "q"), H, K, dk, dv)
    d.num_tokens = T
    d.scale = dk ** -0.5 if scale is None else scale
    _heads(d.q, q, dev, dt, (T, H, dk), "q")
    _heads(d.k, k, dev, dt, (T, K, dk), "k")
    _heads(d.v, v, dev, dt, (T, K, dv), "v")
    d.log_decay = _dense(log_decay, dev, _torch().float32, (H,), "log_decay")
    return d, dev, dt, (T, H, K, dk, dv)


def _sequences(d, dev, cu_seqlens, max_seqlen):
    if cu_seqlens is None:
        d.num_seqs = 1
    else:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        d.num_seqs = cu_seqlens.numel() - 1
        d.cu_seqlens = _dense(cu_seqlens, dev, _torch().int32, cu_seqlens.shape, "cu_seqlens")
    d.max_seqlen = d.num_tokens if max_seqlen is None else int(max_seqlen)
    return d.num_seqs


def linear_attention_workspace(q, k, v, cu_seqlens=None, max_seqlen=None, backward=False):
    """A workspace tensor for pc_linear_attention_forward, or with backward for pc_linear_attention_backward, on
    tensors of these shapes."""
    d, dev, _, _ = _attention(q, k, v, None, None)
    _sequences(d, dev, cu_seqlens, max_seqlen)
    n = _bytes(lib().pc_linear_attention_workspace_bytes, C.byref(d), 1 if backward else 0)
    return _torch().empty(n, dtype=_torch().uint8, device=q.device)


def pc_linear_attention_forward(q, k, v, log_decay, o, cu_seqlens=None, max_seqlen=None, state_in=None, state_out=None,
                                scale=None, ws=None, stream=None):
    """o [tokens, heads, dim_v] from q, k, v along every sequence, S_t = exp(log_decay) S_{t-1} + k_t v_t^T,
    o_t = scale q_t^T S_t.  cu_seqlens: int32 [sequences + 1] on the GPU (None: one sequence); max_seqlen: a bound of
    the longest (None: the number of tokens); states: float32 [sequences, heads, dim_k, dim_v]; scale: None for
    dim_k ** -0.5; ws: linear_attention_workspace(...)."""
    f32 = _torch().float32
    d, dev, dt, (T, H, K, dk, dv) = _attention(q, k, v, log_decay, scale)
    n = _sequences(d, dev, cu_seqlens, max_seqlen)
    _heads(d.o, o, dev, dt, (T, H, dv), "o")
    d.state_in = _dense(state_in, dev, f32, (n, H, dk, dv), "state_in")
    d.state_out = _dense(state_out, dev, f32, (n, H, dk, dv), "state_out")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_linear_attention_forward(dev, d, pws, nws, _stream_of(dev, stream)))


def pc_linear_attention_backward(do, q, k, v, log_decay, dq, dk, dv, cu_seqlens=None, max_seqlen=None, state_in=None,
                                 dstate_out=None, dstate_in=None, scale=None, ws=None, stream=None):
    """dq, dk, dv (and dstate_in) from do (and dstate_out), with the forward call's other arguments;
    ws: linear_attention_workspace(..., backward=True)."""
    f32 = _torch().float32
    d, dev, dt, (T, H, K, nk, nv) = _attention(q, k, v, log_decay, scale)
    n = _sequences(d, dev, cu_seqlens, max_seqlen)
    _heads(d.d_o, do, dev, dt, (T, H, nv), "do")
    _heads(d.d_q, dq, dev, dt, (T, H, nk), "dq")
    _heads(d.d_k, dk, dev, dt, (T, K, nk), "dk")
    _heads(d.d_v, dv, dev, dt, (T, K, nv), "dv")
    d.state_in = _dense(state_in, dev, f32, (n, H, nk, nv), "state_in")
    d.dstate_out = _dense(dstate_out, dev, f32, (n, H, nk, nv), "dstate_out")
    d.dstate_in = _dense(dstate_in, dev, f32, (n, H, nk, nv), "dstate_in")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_linear_attention_backward(dev, d, pws, nws, _stream_of(dev, stream)))


def pc_linear_attention_step(q, k, v, log_decay, state, o, slots=None, scale=None, stream=None):
    """One token for each row of q [rows, heads, dim_k], k, v, o: row b updates state[slots[b]] (slots: int32 [rows] on
    the GPU, None: state[b]) of state [slots, heads, dim_k, dim_v] (float32) in place and reads it.  A slot out of
    range marks a padding row; rows of the same slot are successive tokens, in the rows' order."""
    torch = _torch()
    d, dev, dt, (T, H, K, dk, dv) = _attention(q, k, v, log_decay, scale)
    _heads(d.o, o, dev, dt, (T, H, dv), "o")
    if state.dim() != 4:
        raise ValueError("state must have four dimensions (slots, heads, dim_k, dim_v)")
    d.num_slots = state.shape[0]
    d.state = _dense(state, dev, torch.float32, (d.num_slots, H, dk, dv), "state")
    d.slots = _dense(slots, dev, torch.int32, (T,), "slots")
    _check(lib().pc_linear_attention_step(dev, d, _stream_of(dev, stream)))


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original=0.0, low=1.0, high=32.0,
                       device="cuda"):
    """The pairs' frequencies for pc_rotary_forward: float64 [rotary_dim / 2], base ** (-2 i / rotary_dim) radians a
    position.  scaling, for contexts `factor` times longer than meant: "linear" (all divided by factor), "base" (a larger
    base: the slowest pair is divided by factor), "parts" (pairs of at most `low` turns over `original` positions are
    divided by factor, of at least `high` kept, between them in proportion)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROTARY_SCALINGS)}, got {scaling!r}")
    n = int(rotary_dim)
    host = (C.c_double * max(1, n // 2))()
    _check(lib().pc_rotary_frequencies(n, base, ROTARY_SCALINGS[scaling], factor, original, low, high, host))
    torch = _torch()
    return torch.tensor(list(host)[:n // 2], dtype=torch.float64, device=device)


def _three(t, what):
    if t.dim() != 3:
        raise ValueError(f"{what} must have three dimensions (tokens, heads, dim)")
    return t


def _rotary(q, k, positions, freq, interleaved, magnitude, norm, eps, q_weight, k_weight):
    """The descriptor for heads like q [tokens, heads, dim] and k [tokens, kv_heads, dim] (None: no keys)."""
    torch = _torch()
    dev = _device(_three(q, "q"), "q")
    T, H, dim = q.shape
    d = pc_rotary(_dtype(q, "q"), H, 0 if k is None else _three(k, "k").shape[1], dim, T, 2 * freq.numel(),
                  1 if interleaved else 0, 1 if norm else 0, eps, magnitude)
    d.positions = _dense(positions, dev, torch.int32, (T,), "positions")
    d.freq = _dense(freq, dev, torch.float64, (freq.numel(),), "freq")
    if norm:
        d.q_weight = _dense(q_weight, dev, torch.float32, (dim,), "q_weight")
        d.k_weight = _dense(k_weight, dev, torch.float32, (dim,), "k_weight")
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights belong to the norm: norm is False")
    return d, dev, q.dtype, (T, H, dim), (T, d.kv_heads, dim)


def pc_rotary_forward(q, k, q_out, k_out, positions, freq, interleaved=False, magnitude=1.0, norm=False, q_weight=None,
                      k_weight=None, eps=1e-6, stream=None):
    """q_out, k_out = the heads of q [tokens, heads, dim] and k [tokens, kv_heads, dim] (None: none), normalised by their
    root mean square and weighted (norm; weights: float32 [dim] or None), and turned by positions (int32 [tokens]) times
    freq (rotary_frequencies; its pairs take the first elements, the others are not turned).  Pair i is elements
    (i, i + pairs), interleaved: (2 i, 2 i + 1).  Outputs may be their inputs."""
    d, dev, dt, sq, sk = _rotary(q, k, positions, freq, interleaved, magnitude, norm, eps, q_weight, k_weight)
    _heads(d.q, q, dev, dt, sq, "q")
    _heads(d.q_out, q_out, dev, dt, sq, "q_out")
    if k is not None:
        _heads(d.k, k, dev, dt, sk, "k")
        _heads(d.k_out, k_out, dev, dt, sk, "k_out")
    _check(lib().pc_rotary_forward(dev, d, _stream_of(dev, stream)))


def rotary_workspace(q, k=None):
    """A workspace tensor for pc_rotary_backward with gradients of weights, on heads like q and k."""
    T, H, dim = _three(q, "q").shape
    d = pc_rotary(_dtype(q, "q"), H, 0 if k is None else _three(k, "k").shape[1], dim, T)
    return _torch().empty(_bytes(lib().pc_rotary_workspace_bytes, d), dtype=_torch().uint8, device=q.device)


def pc_rotary_backward(dq_out, dk_out, dq, dk, positions, freq, interleaved=False, magnitude=1.0, norm=False, q=None, k=None,
                       q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, eps=1e-6, ws=None, stream=None):
    """dq, dk from dq_out, dk_out (the gradients of the forward call's outputs), and with norm, from its q and k,
    dq_weight and dk_weight (float32 [dim], overwritten, or None: not wanted).  dq may be dq_out or q, dk likewise.
    ws: rotary_workspace(q, k), needed for the weights' gradients."""
    d, dev, dt, sq, sk = _rotary(dq_out, dk_out, positions, freq, interleaved, magnitude, norm, eps, q_weight, k_weight)
    f32, dim = _torch().float32, sq[2]
    _heads(d.d_q_out, dq_out, dev, dt, sq, "dq_out")
    _heads(d.d_q, dq, dev, dt, sq, "dq")
    if norm:
        _heads(d.q, q, dev, dt, sq, "q")
        d.d_q_weight = _dense(dq_weight, dev, f32, (dim,), "dq_weight")
        d.d_k_weight = _dense(dk_weight, dev, f32, (dim,), "dk_weight")
    elif dq_weight is not None or dk_weight is not None:
        raise ValueError("weights belong to the norm: norm is False")
    if dk_out is not None:
        _heads(d.d_k_out, dk_out, dev, dt, sk, "dk_out")
        _heads(d.d_k, dk, dev, dt, sk, "dk")
        if norm:
            _heads(d.k, k, dev, dt, sk, "k")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_rotary_backward(dev, d, pws, nws, _stream_of(dev, stream)))


def _softmax_attention(q, k, v, scale, cu_seqlens, max_seqlen=None):
    """The descriptor of q [tokens, heads, dim_k], k [tokens, kv_heads, dim_k], v [tokens, kv_heads, dim_v]."""
    dev, dt = _device(_three(q, "q"), "q"), q.dtype
    T, H, dk = q.shape
    K, dv = _three(k, "k").shape[1], _three(v, "v").shape[2]
    d = pc_attention(_dtype(q, "q"), H, K, dk, dv, 1, T)
    d.scale = dk ** -0.5 if scale is None else scale
    d.max_seqlen = T if max_seqlen is None else max_seqlen
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        d.num_seqs = cu_seqlens.numel() - 1
        d.cu_seqlens = _dense(cu_seqlens, dev, _torch().int32, cu_seqlens.shape, "cu_seqlens")
    _heads(d.q, q, dev, dt, (T, H, dk), "q")
    _heads(d.k, k, dev, dt, (T, K, dk), "k")
    _heads(d.v, v, dev, dt, (T, K, dv), "v")
    return d, dev, dt, (T, H, K, dk, dv)


def attention_workspace(q, k, v, cu_seqlens=None, max_seqlen=None, backward=False):
    """A workspace tensor for pc_attention_forward, or with backward for pc_attention_backward, on tensors of these
    shapes and this max_seqlen.  A smaller call can need a larger one (few rows are cut into parts): make one for each shape,
    or take the largest."""
    d, _, _, _ = _softmax_attention(q, k, v, None, cu_seqlens, max_seqlen)
    n = _bytes(lib().pc_attention_workspace_bytes, d, 1 if backward else 0)
    return _torch().empty(n, dtype=_torch().uint8, device=q.device)


def pc_attention_forward(q, k, v, o, lse=None, cu_seqlens=None, max_seqlen=None, scale=None, ws=None, stream=None):
    """Causal softmax attention: o [tokens, heads, dim_v] and lse (float32 [tokens, heads], kept for the backward pass, or
    None) from q, k, v along every sequence.  cu_seqlens: int32 [sequences + 1] on the GPU (None: one sequence);
    max_seqlen: a bound of the longest (None: the number of tokens); scale: None for dim_k ** -0.5;
    ws: attention_workspace(...) (None: keys are not cut into parts, which few long sequences are faster with)."""
    d, dev, dt, (T, H, K, dk, dv) = _softmax_attention(q, k, v, scale, cu_seqlens, max_seqlen)
    _heads(d.o, o, dev, dt, (T, H, dv), "o")
    d.lse = _dense(lse, dev, _torch().float32, (T, H), "lse")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_attention_forward(dev, d, pws, nws, _stream_of(dev, stream)))


def pc_attention_backward(do, q, k, v, o, lse, dq, dk, dv, cu_seqlens=None, max_seqlen=None, scale=None, ws=None, stream=None):
    """dq, dk, dv from do and the forward call's q, k, v, o and lse; ws: attention_workspace(..., backward=True)."""
    d, dev, dt, (T, H, K, nk, nv) = _softmax_attention(q, k, v, scale, cu_seqlens, max_seqlen)
    _heads(d.o, o, dev, dt, (T, H, nv), "o")
    _heads(d.d_o, do, dev, dt, (T, H, nv), "do")
    d.lse = _dense(lse, dev, _torch().float32, (T, H), "lse")
    _heads(d.d_q, dq, dev, dt, (T, H, nk), "dq")
    _heads(d.d_k, dk, dev, dt, (T, K, nk), "dk")
    _heads(d.d_v, dv, dev, dt, (T, K, nv), "dv")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_attention_backward(dev, d, pws, nws, _stream_of(dev, stream)))


def _cached_sizes(d, dev, k_cache, page_table, cu_seqlens, max_seqlen, max_length):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must have four dimensions (pages, page_size, kv_heads, dim_k)")
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dimensions (sequences, pages of each)")
    n = d.num_seqs = page_table.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    d.num_pages, d.page_size, d.max_pages = k_cache.shape[0], k_cache.shape[1], page_table.shape[1]
    d.page_table = _operand(page_table, dev, _torch().int32, (n, d.max_pages), "page_table")
    d.page_table_stride = page_table.stride(0)
    d.max_seqlen = max_seqlen if max_seqlen is not None else 1 if cu_seqlens is None and n > 1 else d.num_tokens
    d.max_length = max_length if max_length is not None else d.max_pages * d.page_size
    return n


def attention_cached_workspace(q, k_cache, v_cache, page_table, cu_seqlens=None, max_seqlen=None, max_length=None):
    """A workspace tensor for pc_attention_cached on new tokens like q and these arguments (as attention_workspace: of these
    shapes and bounds; a smaller call can need a larger one)."""
    T, H, dk = _three(q, "q").shape
    d = pc_attention(_dtype(q, "q"), H, k_cache.shape[2], dk, v_cache.shape[3], 1, T)
    _cached_sizes(d, _device(q, "q"), k_cache, page_table, cu_seqlens, max_seqlen, max_length)
    return _torch().empty(_bytes(lib().pc_attention_cached_workspace_bytes, d), dtype=_torch().uint8, device=q.device)


def _pages(to, t, dev, dtype, shape, what):
    to.data = _operand(t, dev, dtype, shape, what)
    to.page_stride, to.token_stride, to.head_stride, _ = t.stride()


def pc_attention_cached(q, k, v, k_cache, v_cache, page_table, lengths, o, cu_seqlens=None, max_seqlen=None, max_length=None,
                        scale=None, ws=None, stream=None):
    """Causal softmax attention of new tokens over a cache in pages, which they join.  Sequence i has lengths[i] tokens
    (int32 [sequences]) in k_cache [pages, page_size, kv_heads, dim_k] and v_cache, position p in row p % page_size of page
    page_table[i, p // page_size] (int32 [sequences, pages of each]), and the new tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1
    of q, k, v behind them (cu_seqlens None: all of them with one sequence, else one token each).  Writes
    o [tokens, heads, dim_v] and the new tokens' rows of the caches.  max_seqlen, max_length: bounds of a
    sequence's new tokens and of all its tokens (None: those of the shapes); ws: attention_cached_workspace(...) with the same."""
    i32 = _torch().int32
    d, dev, dt, (T, H, K, dk, dv) = _softmax_attention(q, k, v, scale, cu_seqlens)
    n = _cached_sizes(d, dev, k_cache, page_table, cu_seqlens, max_seqlen, max_length)
    _heads(d.o, o, dev, dt, (T, H, dv), "o")
    _pages(d.k_cache, k_cache, dev, dt, (d.num_pages, d.page_size, K, dk), "k_cache")
    _pages(d.v_cache, v_cache, dev, dt, (d.num_pages, d.page_size, K, dv), "v_cache")
    d.cached = _dense(lengths, dev, i32, (n,), "lengths")
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_attention_cached(dev, d, pws, nws, _stream_of(dev, stream)))


def _matrices(t, what):
    """(batch, rows, cols, batch stride, row stride) of a matrix or a batch of them."""
    if t.dim() == 2:
        return 1, t.shape[0], t.shape[1], 0, t.stride(0)
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.shape[2], t.stride(0), t.stride(1)
    raise ValueError(f"{what} must have two or three dimensions")


def orthogonalize_workspace(g):
    """A workspace tensor for pc_orthogonalize on matrices like g."""
    b, r, c, _, _ = _matrices(g, "g")
    n = _bytes(lib().pc_orthogonalize_workspace_bytes, _dtype(g, "g"), b, r, c)
    return _torch().empty(n, dtype=_torch().uint8, device=g.device)


def pc_orthogonalize(g, out, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, ws=None, stream=None):
    """out = the matrices of g [rows, cols] or [batch, rows, cols] after `steps` Newton-Schulz steps from
    g / (|g| + eps), X <- a X + (b A + c A^2) X with A = X X^T; coefficients: (a, b, c), or one such triple for each
    step; out may be g.  ws: orthogonalize_workspace(g)."""
    b, r, c, gb, gr = _matrices(g, "g")
    dev = _device(g, "g")
    pg, po = _operand(g, dev, g.dtype, g.shape, "g"), _operand(out, dev, g.dtype, g.shape, "out")
    _, _, _, ob, orow = _matrices(out, "out")
    steps = int(steps)
    each = list(coefficients)
    if each and not isinstance(each[0], (tuple, list)):
        each = [each] * steps
    if len(each) != steps or any(len(x) != 3 for x in each):
        raise ValueError("coefficients must be (a, b, c) or one such triple for each step")
    flat = (C.c_float * max(1, 3 * steps))(*[float(v) for x in each for v in x])
    pws, nws = _ws_ptr(ws, dev)
    _check(lib().pc_orthogonalize(dev, _dtype(g, "g"), b, r, c, pg, gb, gr, po, ob, orow, steps, flat, eps, pws, nws,
                                  _stream_of(dev, stream)))


class StepGraph:
    """One pass (forward, backward and, with ``em=(step_size, pseudocount)``,
    the EM update) recorded once as a HIP graph on fixed buffers and replayed
    by ``replay()``: every launch of the pass is one graph node, so a replay
    pays no per-launch host cost.  The graph is recorded again when the
    handle's precision mode changed since (the pass's kernels depend on it);
    after any other pc_set_option, make a new StepGraph.  Recording turns the
    handle's per-kernel timing off (its events cannot be graph nodes).  The
    buffers and the workspace must stay allocated, and are read and written in
    place at every replay (a workspace passed in must be large enough for every
    mode the handle will run in: ``workspace(..., all_modes=True)``); ``zero_param_flows`` clears the parameter flows at
    the start of each pass (a fill kernel, not a memset node)."""

    def __init__(self, h: Handle, batch: int, tokens, params, node_vals, node_flows, param_flows,
                 ll=None, flags=0, lowrank=None, grads=None, ws=None, em=None, zero_param_flows=True):
        self.h, self.batch = h, int(batch)
        self.args = (tokens, params, node_vals, node_flows, param_flows, ll, flags, lowrank, grads)
        self.ws = ws if ws is not None else workspace(h, batch, node_vals.device, all_modes=True)
        self.em = em
        self.zero = zero_param_flows
        self.graph = None
        self.mode = None
        # one eager forward + backward first: anything the library sets up on
        # its first call (a second stream for chunked parameter flows) exists
        # before recording; the EM update is left out so parameters do not move
        pc_set_timing(h, False)
        self._pass(None, with_em=False)
        _torch().cuda.synchronize()
        self._record()

    def _pass(self, stream, with_em=True):
        tokens, params, vals, flows, pflows, ll, flags, lowrank, grads = self.args
        s = stream.cuda_stream if stream is not None else None
        if self.zero:
            pflows.zero_()
        pc_forward(self.h, self.batch, tokens, params, vals, ll, lowrank, self.ws, s)
        pc_backward(self.h, self.batch, tokens, params, vals, flows, pflows, flags, lowrank, grads, self.ws, s)
        if with_em and self.em is not None:
            pc_em_step(self.h, params, pflows, self.em[0], self.em[1], s)

    def _record(self):
        torch = _torch()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self._pass(torch.cuda.current_stream())
        self.graph = g
        self.mode = pc_get_precision(self.h)

    def replay(self):
        if pc_get_precision(self.h) != self.mode:
            self._record()
        self.graph.replay()
