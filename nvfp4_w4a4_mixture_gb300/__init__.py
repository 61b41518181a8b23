"""Python binding of libmoe_nvfp4 (include/moe_nvfp4.h): NVFP4 W4A4 routed-MoE layer forward on sm_103a.

Argument marshalling only: every step of the layer runs in the library's CUDA kernels. PyTorch
provides device memory and the current stream. There is no CPU fallback: every call raises if
the shared library is missing or returns an error.
"""
import ctypes
import importlib.machinery
import importlib.util
import os
import sysconfig

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_nvfp4.so")
CALLS_PATH = os.path.join(_HERE, "_lib", "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))

EPI_F32, EPI_BF16, EPI_SWIGLU_NVFP4 = 0, 1, 2
SCHED_AUTO, SCHED_ACT_ON_M, SCHED_WEIGHTS_ON_M, SCHED_WIDE, SCHED_WIDE_ROWS = 0, 0x100, 0x200, 0x400, 0x800
SCHED_WEIGHTS_RESIDENT = 0x1000
DTYPE_BF16, DTYPE_F32 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1

ENTRY_POINTS = (
    "moe_quantize_nvfp4", "moe_quantize_nvfp4_f32", "moe_route_topk", "moe_permute", "moe_prepack_nvfp4",
    "moe_grouped_gemm_nvfp4", "moe_combine", "moe_layer_forward", "moe_layer_forward_profiled", "moe_workspace_bytes",
    "moe_read_device_status", "moe_status_string", "moe_last_error_detail", "moe_route_topk_noalloc",
    "moe_layer_forward_host", "moe_workspace_bytes_host", "moe_layer_workspace_view",
    "moe_set_wait_test_hook", "moe_norm_residual", "moe_select_experts", "moe_adapter_add",
)


class MoeError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__("%s (%s)" % (detail, status))
        self.status = status


class NvFp4Bank(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("gscale", ctypes.c_void_p)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("I", ctypes.c_int),
                ("w_router", ctypes.c_void_p), ("logit_bias", ctypes.c_void_p),
                ("w_gate_up", NvFp4Bank), ("w_down", NvFp4Bank), ("s_mid", ctypes.c_void_p)]


class LayerView(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "bytes", "x_scale", "x_codes", "x_sf", "logits", "logits_ld", "topk_ids", "topk_w", "shared_g",
        "permutation_in_workspace", "expert_offsets", "perm_src", "src_perm", "row_token", "h_codes", "h_sf",
        "h_block_rows", "y", "route_first")]


class NormDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("w_offset", ctypes.c_float), ("residual_scale", ctypes.c_float), ("residual_dtype", ctypes.c_int),
                ("gate", ctypes.c_void_p), ("gate_dtype", ctypes.c_int), ("gate_per_channel", ctypes.c_int),
                ("gate_ld", ctypes.c_int64)]


class RoutingDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("k", ctypes.c_int), ("score", ctypes.c_int), ("n_group", ctypes.c_int),
                ("topk_group", ctypes.c_int), ("group_score", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("scale", ctypes.c_float), ("bias", ctypes.c_void_p)]


class AdaptersDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("r", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


_lib = None
_calls = None  # the C marshalling of the block calls (csrc/calls.c), where it was built


def _load_calls(L):
    global _calls
    _calls = None
    if os.path.exists(CALLS_PATH):
        loader = importlib.machinery.ExtensionFileLoader("_calls", CALLS_PATH)
        try:
            mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
            loader.exec_module(mod)
        except ImportError:  # the same calls go through ctypes
            return
        mod.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (L.moe_norm_residual, L.moe_select_experts, L.moe_adapter_add)),
                 torch.bfloat16, torch.float32, torch.int32)
        _calls = mod


def lib():
    """Load the shared library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_nvfp4.so is not built (%s); run nvfp4_w4a4_mixture_gb300.build.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i32]
        L.moe_last_error_detail.restype = ctypes.c_char_p
        L.moe_last_error_detail.argtypes = []
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.moe_workspace_bytes_host.restype = sz
        L.moe_workspace_bytes_host.argtypes = [i32, i32, i32, i32, i32]
        L.moe_read_device_status.restype = i32
        L.moe_read_device_status.argtypes = [vp, vp]
        for name in ("moe_quantize_nvfp4", "moe_quantize_nvfp4_f32"):
            f = getattr(L, name)
            f.restype = i32
            f.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]
        L.moe_route_topk.restype = i32
        L.moe_route_topk.argtypes = [vp, i32, ctypes.POINTER(LayerDesc), vp, vp, vp, vp, vp, sz, vp]
        L.moe_route_topk_noalloc.restype = i32
        L.moe_route_topk_noalloc.argtypes = [vp, i32, ctypes.POINTER(LayerDesc), vp, vp, vp, vp, vp]
        L.moe_permute.restype = i32
        L.moe_permute.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_prepack_nvfp4.restype = i32
        L.moe_prepack_nvfp4.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
        L.moe_grouped_gemm_nvfp4.restype = i32
        L.moe_grouped_gemm_nvfp4.argtypes = [vp, vp, vp, i32, vp, vp, i32, i64, ctypes.POINTER(NvFp4Bank), i32, i32,
                                             i32, i32, vp, vp, vp, vp, sz, vp]
        L.moe_combine.restype = i32
        L.moe_combine.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
        L.moe_layer_forward.restype = i32
        L.moe_layer_forward.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, vp, vp, vp, sz, vp]
        L.moe_layer_forward_host.restype = i32
        L.moe_layer_forward_host.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, vp, vp, vp, sz, vp]
        L.moe_set_wait_test_hook.restype = i32
        L.moe_set_wait_test_hook.argtypes = [vp, ctypes.c_uint, i32, vp]
        L.moe_layer_workspace_view.restype = i32
        L.moe_layer_workspace_view.argtypes = [ctypes.POINTER(LayerDesc), i32, ctypes.POINTER(LayerView)]
        L.moe_layer_forward_profiled.restype = i32
        L.moe_layer_forward_profiled.argtypes = [ctypes.POINTER(LayerDesc), vp, i32, vp, vp, vp, sz, vp,
                                                 ctypes.POINTER(vp), i32]
        L.moe_norm_residual.restype = i32
        L.moe_norm_residual.argtypes = [ctypes.POINTER(NormDesc), vp, i64, vp, i64, i32, vp, i64, vp, i64, vp]
        L.moe_select_experts.restype = i32
        L.moe_select_experts.argtypes = [ctypes.POINTER(RoutingDesc), vp, i32, i64, i32, vp, vp, vp]
        L.moe_adapter_add.restype = i32
        L.moe_adapter_add.argtypes = [ctypes.POINTER(AdaptersDesc), vp, i64, i32, vp, vp, i32, vp, i64, vp, i64, vp, sz, vp]
        _load_calls(L)
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        L = lib()
        raise MoeError(L.moe_status_string(status).decode(), L.moe_last_error_detail().decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the current stream's handle without a torch.cuda.Stream object (3 us of a call on an Arm host)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def moe_workspace_bytes(H, E, k, I, T):
    return int(lib().moe_workspace_bytes(H, E, k, I, T))


def moe_workspace_bytes_host(H, E, k, I, T):
    return int(lib().moe_workspace_bytes_host(H, E, k, I, T))


class Workspace:
    """Device scratch for the library calls (header zeroed once)."""

    def __init__(self, nbytes, device="cuda"):
        self.nbytes = int(max(nbytes, 4096))
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.buf.data_ptr()) % 256
        self.tensor = self.buf[off: off + self.nbytes]
        self.tensor[:256].zero_()
        self.address = self.tensor.data_ptr()

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())


_default_ws = {}


def _ws(nbytes):
    dev = torch.cuda.current_device()
    w = _default_ws.get(dev)
    if w is None or w.nbytes < nbytes:
        w = Workspace(nbytes)
        _default_ws[dev] = w
    return w


_adapter_ws = {}


def _adapter_workspace():
    """moe_adapter_add's workspace where the caller gives none: its header is all that the call uses, so it is never
    replaced by a larger one, which would lose its report and leave captured calls with memory that was given back."""
    dev = torch.cuda.current_device()
    w = _adapter_ws.get(dev)
    if w is None:
        w = Workspace(4096)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()  # the header is zero for every stream from here on
            _adapter_ws[dev] = w
        # a capture zeroes the header at each replay: its workspace belongs to the graph, and its report is lost
    return w


def moe_set_wait_test_hook(ws, wait_limit_us, ready_extra):
    """Test hook: the expert GEMMs' wait for a token block's intermediate gives up after
    wait_limit_us (0: default) and needs ready_extra more completions (0: none); with more than none,
    moe_adapter_add's wait for A x (long requests) runs out too. (0, 0) restores."""
    _check(lib().moe_set_wait_test_hook(ws.ptr, int(wait_limit_us), int(ready_extra), _stream()))


def moe_read_device_status(ws=None):
    """Raises what the calls on the workspace have reported since the last reading (None: the default workspaces)."""
    if ws is None:
        w = _adapter_ws.get(torch.cuda.current_device())
        if w is not None:
            _check(lib().moe_read_device_status(w.ptr, _stream()))
        ws = _ws(4096)
    _check(lib().moe_read_device_status(ws.ptr, _stream()))


def _bf16_bits(t):
    assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous()
    return t


def moe_quantize_nvfp4(x, s_in=None, ws=None, out=None):
    """x: bf16 or fp32 [rows, K] CUDA tensor -> (codes u8 [rows, K/2], sf u8 [rows, K/16], S f32 [1]).
    out: optional preallocated (codes, sf, s) contiguous views to write into."""
    assert x.is_cuda and x.is_contiguous() and x.dim() == 2
    rows, K = x.shape
    if out is None:
        codes = torch.empty(rows, K // 2, dtype=torch.uint8, device=x.device)
        sf = torch.empty(rows, K // 16, dtype=torch.uint8, device=x.device)
        s_out = torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, sf, s_out = out
        assert codes.is_contiguous() and sf.is_contiguous() and codes.numel() == rows * K // 2
        assert sf.numel() == rows * K // 16
    ws = ws or _ws(4096)
    f = lib().moe_quantize_nvfp4 if x.dtype == torch.bfloat16 else lib().moe_quantize_nvfp4_f32
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be bf16 or fp32")
    _check(f(_p(x), rows, K, _p(s_in), _p(codes), _p(sf), _p(s_out), ws.ptr, ws.nbytes, _stream()))
    return codes, sf, s_out


def moe_prepack_nvfp4(codes, sf, gate_up_interleave):
    """codes u8 [G, N, K/2], sf u8 [G, N, K/16] (row-major) -> prepacked (codes [G, ceil(K/256), N, 128]
    K-slabs, sf tiles)."""
    G, N, Kh = codes.shape
    K = Kh * 2
    codes_out = torch.empty(G, (K + 255) // 256, N, 128, dtype=torch.uint8, device=codes.device)
    sf_out = torch.empty(G * (N // 128) * (K // 64) * 512, dtype=torch.uint8, device=codes.device)
    _check(lib().moe_prepack_nvfp4(_p(codes), _p(sf), G, N, K, int(gate_up_interleave), _p(codes_out), _p(sf_out),
                                   _stream()))
    return codes_out, sf_out


class MoeLayer:
    """Device tensors of one MoE layer plus its C descriptor.

    w_router: bf16 [E+1, H] (row E = shared gate); gate_up: (codes [E+1, 2I, H/2], sf [E+1, 2I, H/16],
    gscale f32 [E+1, 2]) row-major; down: (codes [E+1, H, I/2], sf [E+1, H, I/16], gscale [E+1]);
    s_mid f32 [E+1]; logit_bias nullable f32 [E]. The expert banks are prepacked on the device."""

    def __init__(self, H, E, k, I, w_router, gate_up, down, s_mid, logit_bias=None, prepacked=False):
        self.H, self.E, self.k, self.I = H, E, k, I
        self.w_router = _bf16_bits(w_router)
        if prepacked:
            self.gu_codes, self.gu_sf, self.gu_scale = gate_up
            self.dn_codes, self.dn_sf, self.dn_scale = down
        else:
            self.gu_codes, self.gu_sf = moe_prepack_nvfp4(gate_up[0], gate_up[1], True)
            self.gu_scale = gate_up[2].contiguous()
            self.dn_codes, self.dn_sf = moe_prepack_nvfp4(down[0], down[1], False)
            self.dn_scale = down[2].contiguous()
        self.s_mid = s_mid.contiguous()
        self.logit_bias = logit_bias.contiguous() if logit_bias is not None else None
        self.desc = LayerDesc(H, E, k, I, self.w_router.data_ptr(),
                              self.logit_bias.data_ptr() if self.logit_bias is not None else None,
                              NvFp4Bank(self.gu_codes.data_ptr(), self.gu_sf.data_ptr(), self.gu_scale.data_ptr()),
                              NvFp4Bank(self.dn_codes.data_ptr(), self.dn_sf.data_ptr(), self.dn_scale.data_ptr()),
                              self.s_mid.data_ptr())

    def workspace_bytes(self, T):
        return moe_workspace_bytes(self.H, self.E, self.k, self.I, T)


def moe_route_topk(x, layer, want_logits=False, ws=None):
    T = x.shape[0]
    dev = x.device
    ids = torch.empty(T, layer.k, dtype=torch.int32, device=dev)
    w = torch.empty(T, layer.k, dtype=torch.float32, device=dev)
    g = torch.empty(T, dtype=torch.float32, device=dev)
    lg = torch.empty(T, layer.E, dtype=torch.float32, device=dev) if want_logits else None
    ws = ws or _ws(layer.workspace_bytes(T))
    _check(lib().moe_route_topk(_p(_bf16_bits(x)), T, ctypes.byref(layer.desc), _p(ids), _p(w), _p(g), _p(lg), ws.ptr,
                                ws.nbytes, _stream()))
    return ids, w, g, lg


def moe_permute(topk_ids, E, with_shared=True, ws=None):
    T, k = topk_ids.shape
    dev = topk_ids.device
    offsets = torch.empty(E + 2, dtype=torch.int32, device=dev)
    perm_src = torch.empty(T * k, dtype=torch.int32, device=dev)
    src_perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * k + (T if with_shared else 0), dtype=torch.int32, device=dev)
    ws = ws or _ws(moe_workspace_bytes(128, E, k, 128, T))
    _check(lib().moe_permute(_p(topk_ids.contiguous()), T, k, E, int(with_shared), _p(offsets), _p(perm_src),
                             _p(src_perm), _p(row_token), ws.ptr, ws.nbytes, _stream()))
    return offsets, perm_src, src_perm, row_token


def moe_grouped_gemm_nvfp4(a_codes, a_sf, a_scale, group_offsets, p_max, b_codes, b_sf, b_scale, N, K, gate_up,
                           epilogue, a_row_index=None, epi_scale=None, ws=None, schedule=SCHED_AUTO):
    """Grouped GEMM over a prepacked bank. Returns out (and out_sf for the SwiGLU epilogue)."""
    G = group_offsets.numel() - 1
    dev = a_codes.device
    P = int(p_max)
    out_sf = None
    if epilogue == EPI_F32:
        out = torch.empty(P, N, dtype=torch.float32, device=dev)
    elif epilogue == EPI_BF16:
        out = torch.empty(P, N, dtype=torch.bfloat16, device=dev)
    else:
        out = torch.empty(P, N // 4, dtype=torch.uint8, device=dev)
        out_sf = torch.empty(P, N // 32, dtype=torch.uint8, device=dev)
    bank = NvFp4Bank(b_codes.data_ptr(), b_sf.data_ptr(), b_scale.data_ptr())
    ws = ws or _ws(256 + 4 * (G + 1) + 4096)
    per_group = int(a_scale.numel() > 1)
    _check(lib().moe_grouped_gemm_nvfp4(_p(a_codes), _p(a_sf), _p(a_scale), per_group, _p(a_row_index),
                                        _p(group_offsets), G, P, ctypes.byref(bank), N, K, int(gate_up),
                                        epilogue | schedule,
                                        _p(epi_scale), _p(out), _p(out_sf), ws.ptr, ws.nbytes, _stream()))
    return (out, out_sf) if epilogue == EPI_SWIGLU_NVFP4 else out


def moe_combine(y, topk_w, src_perm, shared_g=None, residual=None):
    T, k = topk_w.shape
    H = y.shape[1]
    out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _check(lib().moe_combine(_p(_bf16_bits(y)), _p(topk_w), _p(shared_g), _p(src_perm), T, k, H,
                             _p(residual), _p(out), _stream()))
    return out


def moe_layer_forward(layer, x, residual=None, out=None, ws=None):
    T = x.shape[0]
    if out is None:
        out = torch.empty(T, layer.H, dtype=torch.bfloat16, device=x.device)
    ws = ws or _ws(layer.workspace_bytes(T))
    _check(lib().moe_layer_forward(ctypes.byref(layer.desc), _p(_bf16_bits(x)), T, _p(residual), _p(out), ws.ptr,
                                   ws.nbytes, _stream()))
    return out


def moe_layer_forward_host(layer, x, residual=None, out=None, ws=None):
    """The layer on host tensors (bf16 [T][H] on the CPU; page-locked keeps the call asynchronous):
    the copies in and out and the layer are enqueued on the current stream. `out` holds the result
    once that stream has passed this call."""
    T = x.shape[0]
    for t in (x, residual, out):
        assert t is None or (t.dtype == torch.bfloat16 and not t.is_cuda and t.is_contiguous())
    if out is None:
        out = torch.empty(T, layer.H, dtype=torch.bfloat16).pin_memory()
    ws = ws or _ws(moe_workspace_bytes_host(layer.H, layer.E, layer.k, layer.I, T))
    _check(lib().moe_layer_forward_host(ctypes.byref(layer.desc), _p(x), T, _p(residual), _p(out), ws.ptr, ws.nbytes,
                                        _stream()))
    return out


def moe_layer_workspace_view(layer, T):
    """The byte offsets of the layer's intermediate results in a forward's workspace (LayerView)."""
    v = LayerView()
    _check(lib().moe_layer_workspace_view(ctypes.byref(layer.desc), T, ctypes.byref(v)))
    return v


def layer_intermediates(layer, T, ws):
    """Views (no copies, no arithmetic) of the intermediate results that the last moe_layer_forward of
    T tokens left in workspace `ws`, at the offsets moe_layer_workspace_view reports. Read them once
    the forward's stream has passed it. Keys: x_scale, x_codes, x_sf, logits [T][E+1] (column E: the
    shared-gate logit), topk_ids, topk_w, shared_g, h_codes, h_sf (tiles), y, route_first (the fused
    router ran before the encoder); with the permutation in the workspace also expert_offsets,
    perm_src, src_perm, row_token."""
    v = moe_layer_workspace_view(layer, T)
    H, E, k, I = layer.H, layer.E, layer.k, layer.I
    buf = ws.tensor
    assert buf.numel() >= v.bytes

    def at(off, nbytes, dtype, shape):
        return buf[off: off + nbytes].view(dtype).reshape(shape)

    P = T * k + T
    n_blocks_max = (P + v.h_block_rows - 1) // v.h_block_rows + E + 1
    out = dict(
        x_scale=at(v.x_scale, 4, torch.float32, (1,)),
        x_codes=at(v.x_codes, T * H // 2, torch.uint8, (T, H // 2)),
        x_sf=at(v.x_sf, T * H // 16, torch.uint8, (T, H // 16)),
        logits=at(v.logits, T * v.logits_ld * 4, torch.float32, (T, v.logits_ld))[:, : E + 1],
        topk_ids=at(v.topk_ids, T * k * 4, torch.int32, (T, k)),
        topk_w=at(v.topk_w, T * k * 4, torch.float32, (T, k)),
        shared_g=at(v.shared_g, T * 4, torch.float32, (T,)),
        h_codes=at(v.h_codes, P * I // 2, torch.uint8, (P, I // 2)),
        h_sf=at(v.h_sf, n_blocks_max * (I // 64) * 512, torch.uint8, (n_blocks_max, I // 64, 512)),
        h_block_rows=int(v.h_block_rows),
        y=at(v.y, P * H * 2, torch.bfloat16, (P, H)),
        permutation_in_workspace=bool(v.permutation_in_workspace),
        route_first=bool(v.route_first),
    )
    if v.permutation_in_workspace:
        out.update(expert_offsets=at(v.expert_offsets, (E + 2) * 4, torch.int32, (E + 2,)),
                   perm_src=at(v.perm_src, T * k * 4, torch.int32, (T * k,)),
                   src_perm=at(v.src_perm, T * k * 4, torch.int32, (T * k,)),
                   row_token=at(v.row_token, P * 4, torch.int32, (P,)))
    return out


LAYER_STAGES = ("quantize", "route", "permute", "experts", "combine")


def moe_layer_forward_profiled(layer, x, events, residual=None, out=None, ws=None):
    """moe_layer_forward recording 6 torch.cuda.Event objects (already created, enable_timing) at the
    stage boundaries of LAYER_STAGES."""
    T = x.shape[0]
    if out is None:
        out = torch.empty(T, layer.H, dtype=torch.bfloat16, device=x.device)
    ws = ws or _ws(layer.workspace_bytes(T))
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record()
    handles = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_layer_forward_profiled(ctypes.byref(layer.desc), _p(_bf16_bits(x)), T, _p(residual), _p(out),
                                            ws.ptr, ws.nbytes, _stream(), handles, len(events)))
    return out


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


_INT_MAX = 0x7FFFFFFF  # of a count in the C calls


def _refuse(t, name, dtype, shape):
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor of %s, got %s on %s" % (name, dtype, t.dtype, t.device))
    if shape[0] > _INT_MAX:
        raise ValueError("%s: %d rows, more than %d" % (name, shape[0], _INT_MAX))
    raise ValueError("%s must have shape %s and be contiguous (rows may be strided where that is allowed), got %s with strides %s"
                     % (name, tuple(shape), tuple(t.shape), t.stride()))


def _whole(t, name, dtype, shape):
    """The data pointer of a contiguous CUDA tensor of that type and shape (an int or None, as ctypes takes it)."""
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous() or shape[0] > _INT_MAX:
        _refuse(t, name, dtype, shape)
    return t.data_ptr()


def _rows(t, name, dtype, shape):
    """(data pointer, elements between two rows) of a CUDA tensor of that type and shape [T, n] whose rows are contiguous."""
    if t.dtype is dtype and t.is_cuda and t.shape == shape and shape[0] <= _INT_MAX:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        if shape[1] == 1 or t.stride(1) == 1:
            return t.data_ptr(), t.stride(0)
    _refuse(t, name, dtype, shape)


def moe_norm_residual(y, residual, w_post=None, w_pre=None, gate=None, residual_scale=1.0, eps=1e-6, w_offset=0.0,
                      out=None):
    """The norm after a block (of its output y, with w_post), its gate, the residual sum and the norm
    before the next block (with w_pre): returns (residual_out, x_out), x_out None without w_pre.

    y: bf16 [T, H] or None; residual: bf16 or fp32 [T, H] or None. gate: bf16 or fp32, [H] (per channel),
    [T, 1] (per token), [T, H] or [1, 1]. out: optional (residual_out, x_out) to write into; a None among
    them is allocated. Rows may be strided."""
    like = y if y is not None else residual
    if like is None:
        raise ValueError("y and residual are both None")
    r_out, x_out = out if out is not None else (None, None)
    if r_out is None:
        r_out = torch.empty(like.shape, dtype=_BF16 if residual is None else residual.dtype, device=like.device)
    if x_out is None and w_pre is not None:
        x_out = torch.empty(like.shape, dtype=_BF16, device=like.device)
    if _lib is None:
        lib()
    status = -1
    if _calls is not None and like.is_cuda:
        status = _calls.norm_residual(y, residual, w_post, w_pre, gate, residual_scale, eps, w_offset, r_out, x_out, _stream())
    if status < 0:
        status = _norm_residual(y, residual, w_post, w_pre, gate, residual_scale, eps, w_offset, r_out, x_out)
    if status:
        _check(status)
    return r_out, x_out


def _norm_residual(y, residual, w_post, w_pre, gate, residual_scale, eps, w_offset, r_out, x_out):
    shape = (y if y is not None else residual).shape
    T, H = shape
    rt = residual.dtype if residual is not None else _BF16
    if rt is not _BF16 and rt is not _F32:
        raise TypeError("residual must be bf16 or fp32, got %s" % rt)
    g_ptr, g_type, g_channel, g_ld = None, 0, 0, 0
    if gate is not None:
        g_shape = gate.shape
        if len(g_shape) == 1:
            gate, g_shape = gate.unsqueeze(0), (1, g_shape[0])
        g_type = DTYPE_F32 if gate.dtype is _F32 else DTYPE_BF16
        g_channel = int(g_shape[1] != 1)
        g_ptr, g_ld = _rows(gate, "gate", _F32 if g_type else _BF16, (1 if g_shape[0] == 1 else T, H if g_channel else 1))
        if g_shape[0] == 1:
            g_ld = 0
    d = NormDesc(H, None if w_post is None else _whole(w_post, "w_post", _BF16, (H,)),
                 None if w_pre is None else _whole(w_pre, "w_pre", _BF16, (H,)), eps, w_offset, residual_scale,
                 DTYPE_F32 if rt is _F32 else DTYPE_BF16, g_ptr, g_type, g_channel, g_ld)
    y_ptr, y_ld = (None, 0) if y is None else _rows(y, "y", _BF16, shape)
    r_ptr, r_ld = (None, 0) if residual is None else _rows(residual, "residual", rt, shape)
    ro_ptr, ro_ld = _rows(r_out, "residual_out", rt, shape)
    x_ptr, x_ld = (None, 0) if x_out is None else _rows(x_out, "x_out", _BF16, shape)
    return lib().moe_norm_residual(d, y_ptr, y_ld, r_ptr, r_ld, T, ro_ptr, ro_ld, x_ptr, x_ld, _stream())


def moe_select_experts(logits, k, bias=None, score=SCORE_SOFTMAX, n_group=1, topk_group=1, group_score=GROUP_MAX,
                       renormalize=True, scale=1.0, out=None):
    """The k experts of each token and their weights from logits [T, E] (bf16 or fp32, rows may be strided):
    (ids int32 [T, k], weights fp32 [T, k]). bias: fp32 [E], for the choice alone. out: optional (ids, weights)."""
    if out is None:
        T = logits.shape[0]
        out = torch.empty(T, k, dtype=_I32, device=logits.device), torch.empty(T, k, dtype=_F32, device=logits.device)
    ids, w = out
    if _lib is None:
        lib()
    status = -1
    if _calls is not None and logits.is_cuda:
        status = _calls.select_experts(logits, k, bias, score, n_group, topk_group, group_score, renormalize, scale, ids, w,
                                       _stream())
    if status < 0:
        if any(not -_INT_MAX <= v <= _INT_MAX for v in (k, score, n_group, topk_group, group_score)):
            raise ValueError("k, score, n_group, topk_group and group_score are ints of 32 bits")
        T, E = logits.shape
        lt = logits.dtype
        l_ptr, l_ld = _rows(logits, "logits", _F32 if lt is _F32 else _BF16, (T, E))
        i_ptr, w_ptr = _whole(ids, "ids", _I32, (T, k)), _whole(w, "weights", _F32, (T, k))
        d = RoutingDesc(E, k, score, n_group, topk_group, group_score, 1 if renormalize else 0, scale,
                        None if bias is None else _whole(bias, "bias", _F32, (E,)))
        status = lib().moe_select_experts(d, l_ptr, DTYPE_F32 if lt is _F32 else DTYPE_BF16, l_ld, T, i_ptr, w_ptr, _stream())
    if status:
        _check(status)
    return ids, w


def moe_adapter_add(x, y, a, b, scale, seg_offsets, seg_adapter, out=None, ws=None):
    """y + scale[i] * (x A_i^T) B_i^T per request, i its adapter (-1: y alone). x bf16 [T, K]; y bf16 [T, N];
    a bf16 [n, r, K]; b bf16 [n, N, r]; scale fp32 [n]; request s has the rows seg_offsets[s] ..
    seg_offsets[s + 1] (int32 [S + 1]) and the adapter seg_adapter[s] (int32 [S]). out: optional, may be y.
    x, y and out may have strided rows. Requests that break the rules are reported by moe_read_device_status(ws)."""
    if out is None:
        out = torch.empty(y.shape, dtype=_BF16, device=y.device)
    if _lib is None:
        lib()
    status = -1
    if x.is_cuda:
        if ws is None:
            ws = _adapter_workspace()
        if _calls is not None:
            status = _calls.adapter_add(x, y, a, b, scale, seg_offsets, seg_adapter, out, ws.address, ws.nbytes, _stream())
    if status < 0:
        T, K = x.shape
        n, r, _ = a.shape
        N, S = y.shape[1], seg_adapter.shape[0]
        x_ptr, x_ld = _rows(x, "x", _BF16, (T, K))
        y_ptr, y_ld = _rows(y, "y", _BF16, (T, N))
        o_ptr, o_ld = _rows(out, "out", _BF16, (T, N))
        d = AdaptersDesc(n, r, K, N, _whole(a, "a", _BF16, (n, r, K)), _whole(b, "b", _BF16, (n, N, r)),
                         _whole(scale, "scale", _F32, (n,)))
        status = lib().moe_adapter_add(d, x_ptr, x_ld, T, _whole(seg_offsets, "seg_offsets", _I32, (S + 1,)),
                                       _whole(seg_adapter, "seg_adapter", _I32, (S,)), S, y_ptr, y_ld, o_ptr, o_ld,
                                       ws.address, ws.nbytes, _stream())
    if status:
        _check(status)
    return out
