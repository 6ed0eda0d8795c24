"""Python binding of libgptq (ctypes).  Argument marshalling only: every step of the
solve runs in the library's CUDA kernels; PyTorch provides device memory and the stream.

The object mirrors the three-call lifecycle of the GPTQ quantizer on the page
"模型量化实战：从 INT8 PTQ 到 GPTQ 的精度保持与推理加速全解析" (§3.2: accumulate the Hessian
over calibration batches, prepare the inverse factor, quantize the layer), with the
quantizer settings named as in AutoGPTQ's quantize_config ("GPTQ算法原理深度解析" §3.3).
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gptq.h")
HEADERS = [HEADER, os.path.join(os.path.dirname(HERE), "include", "gptq_testing.h")]

STATUS = {0: "GPTQ_OK", 1: "GPTQ_ERR_ARG", 2: "GPTQ_ERR_STATE", 3: "GPTQ_ERR_NOT_PD", 4: "GPTQ_ERR_OOM",
          5: "GPTQ_ERR_CUDA", 6: "GPTQ_ERR_TIMEOUT", 7: "GPTQ_ERR_UNSUPPORTED"}
OK, ERR_ARG, ERR_STATE, ERR_NOT_PD, ERR_OOM, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED = range(8)


class GPTQError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{call}: {self.name} ({lib().gptq_status_string(status).decode()})")


class QParams(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group_size", ctypes.c_int), ("sym", ctypes.c_int)]


class LayerJob(ctypes.Structure):
    _fields_ = [("X_bf16", ctypes.c_void_p), ("n_tok", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("W_fp16", ctypes.c_void_p), ("m", ctypes.c_int64), ("n", ctypes.c_int64), ("qp", QParams),
                ("damp", ctypes.c_double), ("desc_act", ctypes.c_int), ("codes_out", ctypes.c_void_p),
                ("scales_out", ctypes.c_void_p), ("zeros_out", ctypes.c_void_p), ("g_idx_out", ctypes.c_void_p),
                ("perm_out", ctypes.c_void_p), ("W_hat_out", ctypes.c_void_p)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int64), ("ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


# Argument blocks of the calls on packed layers (the C structures of the same names), packed natively;
# "0q" pads to the alignment of the nested structure's end.
_PACKED = "PPPPqqiii0q"                                                    # gptq_packed
_LINEAR_ARGS = struct.Struct("@Pqqi0q" + _PACKED + "PPqiPqiPPN")           # gptq_linear_args
_LINEAR_GRAD_ARGS = struct.Struct("@Pqqi0q" + _PACKED + "iPPqPPN")         # gptq_linear_grad_args
_MOE_ARGS = struct.Struct("@PqqiPqiii0q" + _PACKED + _PACKED + "PqPqPPPN")  # gptq_moe_args


ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = range(4)
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}

_LIB = None
_P = ctypes.c_void_p
_SIGS = {
    "gptq_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "gptq_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _P]),
    "gptq_hessian_accumulate": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int64]),
    "gptq_get_hessian": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int64)]),
    "gptq_set_hessian": (ctypes.c_int, [_P, _P, ctypes.c_int64]),
    "gptq_prepare": (ctypes.c_int, [_P, ctypes.c_double, ctypes.c_int, _P]),
    "gptq_get_factor": (ctypes.c_int, [_P, _P]),
    "gptq_quantize_layer": (ctypes.c_int, [_P, _P, ctypes.c_int64, QParams, _P, _P, _P, _P, _P]),
    "gptq_synchronize": (ctypes.c_int, [_P]),
    "gptq_reset": (ctypes.c_int, [_P]),
    "gptq_destroy": (ctypes.c_int, [_P]),
    "gptq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gptq_set_hessian_chunk": (ctypes.c_int, [_P, ctypes.c_int64]),
    "gptq_launch_count": (ctypes.c_int64, [_P]),
    "gptq_get_dead_columns": (ctypes.c_int, [_P, _P]),
    "gptq_set_profiling": (ctypes.c_int, [_P, ctypes.c_int]),
    "gptq_get_profile": (ctypes.c_int, [_P, ctypes.POINTER(KernelStat), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
    "gptq_test_bounded_wait": (ctypes.c_int, [_P, ctypes.c_uint64]),
    "gptq_dequant_matmul_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                              ctypes.c_int]),
    "gptq_dequant_matmul": (ctypes.c_int, [_P, ctypes.c_int64, _P, _P, _P, _P, ctypes.c_int64, ctypes.c_int64,
                                           QParams, _P, _P, ctypes.c_size_t, ctypes.c_int, _P]),
    "gptq_dequant_matmul_check": (ctypes.c_int, [_P, ctypes.c_int, _P]),
    "gptq_dequant_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "gptq_dequant_linear": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_int, _P]),
    "gptq_dequant_linear_backward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                                       ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                                       ctypes.c_int]),
    "gptq_dequant_linear_backward": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_int, _P]),
    "gptq_dequant_moe_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                                           ctypes.c_int64, ctypes.c_int64]),
    "gptq_dequant_moe": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_int, _P]),
    "gptq_quantize_layers": (ctypes.c_int, [ctypes.POINTER(LayerJob), ctypes.c_int, ctypes.c_int, _P]),
    "gptq_pipeline_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int64),
                                            ctypes.POINTER(ctypes.c_int64), ctypes.c_int, ctypes.c_int, _P]),
    "gptq_pipeline_run": (ctypes.c_int, [_P, ctypes.POINTER(LayerJob), ctypes.c_int]),
    "gptq_pipeline_destroy": (ctypes.c_int, [_P]),
    "gptq_activation_convert": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int, _P, _P, ctypes.c_int,
                                               _P]),
    "gptq_awq_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64]),
    "gptq_awq_quantize": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_float, QParams, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                         ctypes.c_int, _P]),
    "gptq_rtn_quantize": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, QParams, ctypes.c_float, _P, _P, _P, _P,
                                         _P, ctypes.c_int, _P]),
    "gptq_quantize_layer_noalloc": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, QParams,
                                                   _P, _P, _P, _P, _P, ctypes.c_int, _P]),
    "gptq_test_gemm_tf32x3": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, _P, _P, ctypes.c_int, _P, _P,
                                             ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, _P, ctypes.c_int, _P, _P, ctypes.c_int, _P, _P,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             _P]),
    "gptq_test_div_rn": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_int64, ctypes.POINTER(ctypes.c_uint64),
                                        ctypes.POINTER(ctypes.c_float), ctypes.c_int, _P]),
    "gptq_test_pick_tile_n": (ctypes.c_int, [ctypes.c_int] * 7),
    "gptq_test_tile_schedule": (ctypes.c_int, [ctypes.c_int] * 8),
    "gptq_test_factor_plan": (ctypes.c_int, [ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_int)]),
    "gptq_test_pct_position": (ctypes.c_int, [ctypes.c_double, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                              ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float),
                                              ctypes.POINTER(ctypes.c_float)]),
}


def lib():
    """Load libgptq.so (built in-tree).  Fails loudly when it is missing: there is no fallback."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgptq.so is not built ({LIB_PATH}); run "
                               "`python -m post_weight_quantization_16_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def header_functions():
    """Names of the functions the headers under include/ declare."""
    names = set()
    for h in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names |= set(re.findall(r"\b(gptq_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def _check(status: int, call: str):
    if status != OK:
        raise GPTQError(status, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class GPTQContext:
    """One layer width n: accumulate H over calibration batches, prepare, quantize layers."""

    def __init__(self, n: int, m_max: int, device: int | torch.device = 0, stream: torch.cuda.Stream | None = None):
        self.device = torch.device("cuda", device if isinstance(device, int) else device.index)
        self.n, self.m_max = int(n), int(m_max)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        h = ctypes.c_void_p()
        _check(lib().gptq_create(ctypes.byref(h), self.n, self.m_max, self.device.index,
                                 ctypes.c_void_p(self.stream.cuda_stream)), "gptq_create")
        self._h = h

    # -- lifecycle ---------------------------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            st = lib().gptq_destroy(self._h)
            self._h = None
            _check(st, "gptq_destroy")

    def __del__(self):
        try:
            if getattr(self, "_h", None):
                lib().gptq_destroy(self._h)
                self._h = None
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # -- S1 ----------------------------------------------------------------------------------
    def set_hessian_chunk(self, tokens: int):
        _check(lib().gptq_set_hessian_chunk(self._h, int(tokens)), "gptq_set_hessian_chunk")

    def accumulate_hessian(self, X: torch.Tensor):
        """H += 2 X^T X for a bf16 batch X [tokens, n] on the device (row stride may exceed n)."""
        if X.dtype != torch.bfloat16 or X.device != self.device or X.dim() != 2 or X.stride(1) != 1:
            raise ValueError("X must be a bf16 [tokens, n] device tensor with unit column stride")
        _check(lib().gptq_hessian_accumulate(self._h, _ptr(X), X.shape[0], X.stride(0)), "gptq_hessian_accumulate")

    def get_hessian(self):
        H = torch.empty((self.n, self.n), dtype=torch.float32, device=self.device)
        nt = ctypes.c_int64()
        _check(lib().gptq_get_hessian(self._h, _ptr(H), ctypes.byref(nt)), "gptq_get_hessian")
        return H, nt.value

    def set_hessian(self, H: torch.Tensor, n_tok: int):
        if H.dtype != torch.float32 or H.shape != (self.n, self.n) or not H.is_contiguous() or H.device != self.device:
            raise ValueError("H must be a contiguous fp32 [n, n] device tensor")
        _check(lib().gptq_set_hessian(self._h, _ptr(H), int(n_tok)), "gptq_set_hessian")

    # -- S2-S4 -------------------------------------------------------------------------------
    def prepare(self, damp: float = 0.01, desc_act: bool = False) -> torch.Tensor:
        perm = torch.empty(self.n, dtype=torch.int32, device=self.device)
        _check(lib().gptq_prepare(self._h, float(damp), int(bool(desc_act)), _ptr(perm)), "gptq_prepare")
        return perm

    def get_dead_columns(self) -> torch.Tensor:
        """uint8 [n] mask (original column order) of the columns the last prepare found unexcited."""
        d = torch.empty(self.n, dtype=torch.uint8, device=self.device)
        _check(lib().gptq_get_dead_columns(self._h, _ptr(d)), "gptq_get_dead_columns")
        return d

    def get_factor(self) -> torch.Tensor:
        U = torch.empty((self.n, self.n), dtype=torch.float32, device=self.device)
        _check(lib().gptq_get_factor(self._h, _ptr(U)), "gptq_get_factor")
        return U

    # -- S5-S7 -------------------------------------------------------------------------------
    def quantize_layer(self, W: torch.Tensor, bits: int = 4, group_size: int = 128, sym: bool = False,
                       want_w_hat: bool = True, out: dict | None = None) -> dict:
        """Quantize fp16 W [m, n] (original column order).  Returns device tensors
        codes [m, n*bits/32] int32-viewed uint32 words, scales/zeros [m, G], g_idx [n], w_hat [m, n]."""
        if W.dtype != torch.float16 or W.dim() != 2 or W.shape[1] != self.n or not W.is_contiguous() \
                or W.device != self.device:
            raise ValueError("W must be a contiguous fp16 [m, n] device tensor")
        m = W.shape[0]
        g = self.n if group_size == -1 else group_size
        G = self.n // g if g > 0 and self.n % g == 0 else 1
        if out is None:
            out = {
                "codes": torch.empty((m, self.n * bits // 32), dtype=torch.int32, device=self.device),
                "scales": torch.empty((m, G), dtype=torch.float32, device=self.device),
                "zeros": torch.empty((m, G), dtype=torch.float32, device=self.device),
                "g_idx": torch.empty(self.n, dtype=torch.int32, device=self.device),
                "w_hat": torch.empty((m, self.n), dtype=torch.float32, device=self.device) if want_w_hat else None,
            }
        qp = QParams(int(bits), int(group_size), int(bool(sym)))
        _check(lib().gptq_quantize_layer(self._h, _ptr(W), m, qp, _ptr(out["codes"]), _ptr(out["scales"]),
                                         _ptr(out["zeros"]), _ptr(out["g_idx"]), _ptr(out.get("w_hat"))),
               "gptq_quantize_layer")
        return out

    def synchronize(self):
        _check(lib().gptq_synchronize(self._h), "gptq_synchronize")

    # -- instrumentation ---------------------------------------------------------------------
    def set_profiling(self, on: bool):
        _check(lib().gptq_set_profiling(self._h, int(bool(on))), "gptq_set_profiling")

    def get_profile(self) -> dict:
        """{role: {"launches", "ms", "flops", "bytes"}} of the launches recorded since the last call."""
        cap = 64
        arr = (KernelStat * cap)()
        cnt = ctypes.c_int()
        _check(lib().gptq_get_profile(self._h, arr, cap, ctypes.byref(cnt)), "gptq_get_profile")
        return {arr[i].name.decode(): {"launches": int(arr[i].launches), "ms": arr[i].ms, "flops": arr[i].flops,
                                      "bytes": arr[i].bytes} for i in range(min(cap, cnt.value))}

    def launch_count(self) -> int:
        return int(lib().gptq_launch_count(self._h))

    def reset(self):
        _check(lib().gptq_reset(self._h), "gptq_reset")


def allreduce_hessian(ctx, group=None) -> int:
    """Token-split calibration across the ranks of a torch.distributed group: each rank has
    accumulated 2 X^T X over its own share of the tokens ("模型量化实战…" §3.2 accumulate_hessian:
    the Hessian is a sum over tokens, so partial sums add).  The partial H and token counts are
    summed with one all-reduce each (n^2 fp32 on the group's backend: NCCL over NVLink between
    GPUs) and every rank's context continues from the full H.  Returns the total token count.
    Every rank must call it, in the same order as its other collectives."""
    import torch.distributed as dist
    H, nt = ctx.get_hessian()
    dist.all_reduce(H, op=dist.ReduceOp.SUM, group=group)
    t = torch.tensor([nt], dtype=torch.int64, device=H.device)
    dist.all_reduce(t, op=dist.ReduceOp.SUM, group=group)
    total = int(t.item())
    ctx.set_hessian(H, total)
    return total


def workspace_bytes(n: int, m_max: int) -> int:
    return int(lib().gptq_workspace_bytes(int(n), int(m_max)))


def dequant_matmul(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                   perm: torch.Tensor | None, bits: int, group_size: int, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Y = X W16^T from the packed result (gptq_dequant_matmul).  X: fp16 [T, n] device tensor in
    original column order; codes/scales/zeros as gptq_quantize_layer wrote them; perm or None.
    Returns fp32 Y [T, m] (asynchronous on `stream`)."""
    if X.dtype != torch.float16 or X.dim() != 2 or not X.is_contiguous():
        raise ValueError("X must be a contiguous fp16 [T, n] device tensor")
    T, n = X.shape
    m = codes.shape[0]
    dev = X.device
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    need = int(lib().gptq_dequant_matmul_workspace_bytes(T, m, n, int(perm is not None)))
    if need == 0:
        raise GPTQError(ERR_ARG, "gptq_dequant_matmul_workspace_bytes")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((T, m), dtype=torch.float32, device=dev)
    qp = QParams(int(bits), int(group_size), 0)
    _check(lib().gptq_dequant_matmul(_ptr(X), T, _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(perm), m, n, qp,
                                     _ptr(out), _ptr(workspace), workspace.numel(), dev.index,
                                     ctypes.c_void_p(stream.cuda_stream)), "gptq_dequant_matmul")
    return out


def _packed(codes, scales, zeros, perm, bits: int, group_size: int, index: int, experts: int = 0) -> tuple:
    """Fields of gptq_packed for a packed layer (`experts`: that many stacked ones), its tensors checked."""
    lead = (experts,) if experts else ()
    shape = codes.shape
    if len(shape) != 2 + len(lead) or (experts and shape[0] != experts):
        raise ValueError(f"codes must be {'[E, m, words]' if lead else '[m, words]'}, got {tuple(shape)}")
    m, words = shape[-2], shape[-1]
    n, rest = divmod(words * 32, bits) if bits in (2, 3, 4, 8) else (0, 1)
    if rest or n == 0:
        raise ValueError(f"bits must be 2, 3, 4 or 8 and fit the rows of codes, got {bits}")
    g = n if group_size == -1 else group_size
    if g < 32 or n % g:
        raise ValueError(f"group_size {group_size} does not divide {n} columns")
    want = (*lead, m, n // g)
    for name, t, dt, sh in (("codes", codes, torch.int32, shape), ("scales", scales, torch.float32, want),
                            ("zeros", zeros, torch.float32, want)):
        if t.dtype is not dt or t.shape != sh or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} {tuple(sh)} tensor on cuda:{index}")
    p = None
    if perm is not None:
        if perm.dtype is not torch.int32 or perm.shape != (*lead, n) or perm.get_device() != index \
                or not perm.is_contiguous():
            raise ValueError(f"perm must be a contiguous torch.int32 {(*lead, n)} tensor on cuda:{index}")
        p = perm.data_ptr()
    return codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), p or 0, m, n, bits, group_size, 0


def _rows(name: str, t: torch.Tensor | None, rows: int, cols: int, dtype: torch.dtype, index: int) -> tuple:
    """(pointer, row stride) of an optional row-major matrix with unit column stride."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != index or (t.stride(1) != 1 and cols > 1):
        raise ValueError(f"{name} must be a {dtype} {(rows, cols)} tensor with unit column stride on cuda:{index}")
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _activations(name: str, X: torch.Tensor, n: int) -> tuple:
    """Checks of the left operand: (pointer, tokens, row stride, dtype code)."""
    shape = X.shape
    if len(shape) != 2 or shape[1] != n or X.dtype not in _DTYPES or not X.is_cuda or (X.stride(1) != 1 and n > 1):
        raise ValueError(f"{name} must be an fp16 or bf16 [T, {n}] device tensor with unit column stride")
    T = shape[0]
    ld, at = (X.stride(0) if T > 1 else n), X.data_ptr()
    if ld % 8 or ld < n or at % 16:
        raise ValueError(f"{name} needs a 16-byte aligned base and a row stride that is a multiple of 8 elements "
                         "and no smaller than a row")
    return at, T, ld, _DTYPES[X.dtype]


# The current stream's handle without building a Stream object, where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(stream, like: torch.Tensor) -> bool:
    """Whether `stream` is given and not the current one of the tensor's device."""
    if stream is None:
        return False
    if stream.device_index != like.get_device():
        raise ValueError(f"stream belongs to cuda:{stream.device_index}, the tensors to {like.device}")
    return stream.cuda_stream != _raw_stream(stream.device_index)


class _On:
    """Allocations and launches of a call on a stream that is not the current one."""

    def __init__(self, stream: torch.cuda.Stream):
        self.ctx = torch.cuda.stream(stream)
        self.handle = stream.cuda_stream

    def __enter__(self):
        self.ctx.__enter__()
        return self.handle

    def __exit__(self, *a):
        self.ctx.__exit__(*a)


def _workspace(need: int, workspace: torch.Tensor | None, like: torch.Tensor) -> torch.Tensor:
    """The caller's workspace, checked, or a new one of `need` bytes on the device of `like`."""
    if need == 0:
        raise GPTQError(ERR_ARG, "workspace size")
    if workspace is None:
        return like.new_empty(need, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or workspace.device != like.device or not workspace.is_contiguous() \
            or workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {like.device}")
    return workspace


def check_workspace(workspace: torch.Tensor, stream: torch.cuda.Stream | None = None):
    """Wait (bounded) for `stream` (default: the workspace's device's current one) and raise GPTQError with
    status ERR_TIMEOUT if a bounded wait of the last dequant_matmul, dequant_linear, dequant_linear_backward
    or dequant_moe on this workspace ran out: its outputs are then not to be used.  (A call without tokens
    leaves the workspace as it was.)  Not while a graph is captured; after a replay it tells of that."""
    index = workspace.get_device()
    if index < 0 or workspace.dtype != torch.uint8 or workspace.numel() < 256:
        raise ValueError("workspace must be a uint8 device tensor that a call was given")
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(lib().gptq_dequant_matmul_check(workspace.data_ptr(), index, handle), "a call on this workspace")


def dequant_linear(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                   perm: torch.Tensor | None, bits: int, group_size: int, bias: torch.Tensor | None = None,
                   act: int = ACT_NONE, residual: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                   want_preact: bool = False, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None, check: bool = False):
    """Y = act(X[:, perm] W^T + bias) + residual with a packed W (gptq_dequant_linear).  X: fp16 or
    bf16 [T, n] device tensor in original column order (row stride a multiple of 8); codes, scales,
    zeros, perm as quantize_layer (or rtn_quantize: perm None) wrote them (the product is with the scaled
    weight where the layer has a channel_scale, as awq_quantize's: divide X by it before, and dX after
    dequant_linear_backward); bias [m] and residual [T, m] in X's type; act one of ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU.  Returns Y [T, m]
    in X's type (or fp32 with out_dtype=torch.float32), and with want_preact also Z, the value the
    activation was applied to, which dequant_linear_backward takes.  `out` may be `residual`,
    but not share memory with X.
    Asynchronous on `stream` (default: the device's current one; another stream's allocations are made
    on it); can be captured into a graph.  check: wait for the call and raise if one of its bounded waits
    ran out (check_workspace does that for a caller's workspace, later or after a graph's replay).  Records
    no autograd graph: Y does not require a gradient, dequant_linear_backward is the call for it."""
    if _elsewhere(stream, X):
        with _On(stream):
            return dequant_linear(X, codes, scales, zeros, perm, bits, group_size, bias, act, residual, out_dtype,
                                  want_preact, out, workspace, check=check)
    index = X.get_device()
    W = _packed(codes, scales, zeros, perm, bits, group_size, index)
    m, n = W[4], W[5]
    x_ptr, T, ldx, dt = _activations("X", X, n)
    xt = X.dtype
    b_ptr = 0
    if bias is not None:
        if bias.dtype is not xt or bias.shape != (m,) or bias.get_device() != index or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous {xt} [{m}] tensor on cuda:{index}")
        b_ptr = bias.data_ptr()
    r_ptr, ldr = _rows("residual", residual, T, m, xt, index)
    if out_dtype is None or out_dtype is xt:
        y_type, f32 = xt, 0
    elif out_dtype is torch.float32:
        y_type, f32 = out_dtype, 1
    else:
        raise ValueError("out_dtype must be X's type or torch.float32")
    if out is None:
        out = X.new_empty((T, m), dtype=y_type) if f32 else X.new_empty((T, m))
        y_ptr, ldy = out.data_ptr(), m
    else:
        y_ptr, ldy = _rows("out", out, T, m, y_type, index)
    z = X.new_empty((T, m)) if want_preact else None
    L = lib()
    ws = _workspace(L.gptq_dequant_linear_workspace_bytes(T, n, perm is not None), workspace, X)
    a = _LINEAR_ARGS.pack(x_ptr, T, ldx, dt, *W, b_ptr, r_ptr, ldr, act, y_ptr, ldy, f32, 0 if z is None else z.data_ptr(),
                          ws.data_ptr(), ws.numel())
    st = L.gptq_dequant_linear(a, index, _raw_stream(index))
    if st != OK:
        raise GPTQError(st, "gptq_dequant_linear")
    if check and T:
        check_workspace(ws)
    return (out, z) if want_preact else out


def dequant_linear_backward(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                            perm: torch.Tensor | None, bits: int, group_size: int, act: int = ACT_NONE,
                            preact: torch.Tensor | None = None, want_dx: bool = True, want_dbias: bool = False,
                            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None, check: bool = False):
    """The gradient of dequant_linear with W frozen (gptq_dequant_linear_backward).  dY: fp16 or bf16
    [T, m]; preact: the Z that dequant_linear(want_preact=True) gave (needed unless act is ACT_NONE).
    Returns dX [T, n] in dY's type, or (dX, dbias) with want_dbias (dbias fp32 [m]; dX is None with
    want_dx=False).  The residual's gradient is dY itself.  Asynchronous on `stream`; check as in
    dequant_linear."""
    if _elsewhere(stream, dY):
        with _On(stream):
            return dequant_linear_backward(dY, codes, scales, zeros, perm, bits, group_size, act, preact, want_dx,
                                           want_dbias, out, workspace, check=check)
    index = dY.get_device()
    W = _packed(codes, scales, zeros, perm, bits, group_size, index)
    m, n = W[4], W[5]
    if dY.dim() != 2 or dY.shape[1] != m or dY.dtype not in _DTYPES or not dY.is_cuda:
        raise ValueError(f"dY must be an fp16 or bf16 [T, {m}] device tensor")
    T, t = dY.shape[0], dY.dtype
    dy_ptr, ld_dy = _rows("dY", dY, T, m, t, index)
    z_ptr = 0
    if act != ACT_NONE:
        if preact is None or preact.dtype is not t or preact.shape != (T, m) or not preact.is_contiguous() \
                or preact.get_device() != index:
            raise ValueError(f"preact must be a contiguous {t} [{T}, {m}] tensor on cuda:{index}")
        z_ptr = preact.data_ptr()
    if not (want_dx or want_dbias):
        raise ValueError("nothing to compute: want_dx and want_dbias are both off")
    dt = _DTYPES[t]
    dx = (dY.new_empty((T, n)) if out is None else out) if want_dx else None
    dx_ptr, ld_dx = _rows("out", dx, T, n, t, index)
    db = dY.new_empty(m, dtype=torch.float32) if want_dbias else None
    L = lib()
    ws = _workspace(L.gptq_dequant_linear_backward_workspace_bytes(T, m, n, perm is not None, dt, act), workspace, dY)
    a = _LINEAR_GRAD_ARGS.pack(dy_ptr, T, ld_dy, dt, *W, act, z_ptr, dx_ptr, ld_dx, 0 if db is None else db.data_ptr(),
                               ws.data_ptr(), ws.numel())
    st = L.gptq_dequant_linear_backward(a, index, _raw_stream(index))
    if st != OK:
        raise GPTQError(st, "gptq_dequant_linear_backward")
    if check and T:
        check_workspace(ws)
    return (dx, db) if want_dbias else dx


def dequant_moe(X: torch.Tensor, router: torch.Tensor, gate_up: tuple, down: tuple, perm: torch.Tensor | None,
                bits: int, group_size: int, top_k: int, renormalize: bool = True, act: int = ACT_SILU,
                residual: torch.Tensor | None = None, down_group_size: int | None = None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None, check: bool = False):
    """The mixture-of-experts layer for at most 128 tokens on packed experts (gptq_dequant_moe).
    X: fp16 or bf16 [T, H]; router [E, H] in X's type; gate_up = (codes [E, 2 I, words], scales, zeros)
    with the gate rows first; down = (codes [E, H, words], scales, zeros); perm: int32 [E, H], the
    act-order of each expert's gate and up, or None (stack_experts builds these from quantized
    layers).  Returns Y [T, H], the chosen experts [T, top_k] (int32, by descending probability) and
    their weights [T, top_k] (fp32).  `out` may be X or `residual`.  Asynchronous on `stream`; check as in
    dequant_linear."""
    if _elsewhere(stream, X):
        with _On(stream):
            return dequant_moe(X, router, gate_up, down, perm, bits, group_size, top_k, renormalize, act, residual,
                               down_group_size, out, workspace, check=check)
    index = X.get_device()
    E = router.shape[0] if router.dim() == 2 else 0
    if E == 0:
        raise ValueError("router must be [E, H] with at least one expert")
    gu = _packed(*gate_up, perm, bits, group_size, index, E)
    dn = _packed(*down, None, bits, group_size if down_group_size is None else down_group_size, index, E)
    H, I = gu[5], dn[5]
    if gu[4] != 2 * I or dn[4] != H:
        raise ValueError(f"gate_up [E, {gu[4]}, {H} columns] and down [E, {dn[4]}, {I} columns] do not fit together")
    x_ptr, T, ldx, dt = _activations("X", X, H)
    if router.dtype is not X.dtype or router.shape[1] != H or not router.is_contiguous() or router.get_device() != index:
        raise ValueError(f"router must be a contiguous {X.dtype} [E, {H}] tensor on cuda:{index}")
    r_ptr, ldr = _rows("residual", residual, T, H, X.dtype, index)
    if out is None:
        out = X.new_empty((T, H))
    y_ptr, ldy = _rows("out", out, T, H, X.dtype, index)
    L = lib()
    ws = _workspace(L.gptq_dequant_moe_workspace_bytes(T, E, top_k, H, I), workspace, X)
    ids = X.new_empty((T, top_k), dtype=torch.int32)
    weights = X.new_empty((T, top_k), dtype=torch.float32)
    a = _MOE_ARGS.pack(x_ptr, T, ldx, dt, router.data_ptr(), E, top_k, renormalize, act, *gu, *dn, r_ptr, ldr, y_ptr, ldy,
                       ids.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel())
    st = L.gptq_dequant_moe(a, index, _raw_stream(index))
    if st != OK:
        raise GPTQError(st, "gptq_dequant_moe")
    if check and T:
        check_workspace(ws)
    return out, ids, weights


def stack_experts(gates: list, ups: list, downs: list) -> tuple:
    """(gate_up, down, perm) for dequant_moe from the experts' quantized projections: lists, one entry
    per expert, of dicts with codes, scales, zeros and perm (or no perm) as quantize_layer and
    rtn_quantize return them.  A layer with a channel_scale other than 1 (awq_quantize, rtn_quantize given
    one) is refused: its codes are those of the scaled weight, and dequant_moe has no place where an
    expert's input could be divided by it.  An expert's gate and up share their input, so with
    act-order they must share their perm too (it depends on the input alone).  The act-order of a down
    projection is folded into the rows of its gate and up: h then comes out in down's sweep order.
    A one-time layout: call it once per layer and keep the result."""
    if not gates or len(gates) != len(ups) or len(gates) != len(downs):
        raise ValueError("gates, ups and downs need one entry per expert each")
    gate_up, down, perms = [], [], []
    for e, (g, u, d) in enumerate(zip(gates, ups, downs)):
        for name, q in (("gate", g), ("up", u), ("down", d)):
            c = q.get("channel_scale")
            if c is not None and not bool((c == 1).all()):
                raise ValueError(f"expert {e}: {name} has a channel_scale, which dequant_moe cannot divide out")
        pg, pu, pd = g.get("perm"), u.get("perm"), d.get("perm")
        if (pg is None) != (pu is None) or (pg is not None and not torch.equal(pg, pu)):
            raise ValueError(f"expert {e}: gate and up have different input orders")
        rows = (lambda t: t) if pd is None else (lambda t, i=pd.long(): t.index_select(0, i))
        gate_up.append([torch.cat([rows(g[k]), rows(u[k])]) for k in ("codes", "scales", "zeros")])
        down.append([d[k] for k in ("codes", "scales", "zeros")])
        perms.append(pg)
    if any((p is None) != (perms[0] is None) for p in perms):
        raise ValueError("either every expert has an input order or none has")
    return (tuple(torch.stack(t) for t in zip(*gate_up)), tuple(torch.stack(t) for t in zip(*down)),
            None if perms[0] is None else torch.stack(perms))


def _jobs(layers: list, dev: torch.device):
    jobs = (LayerJob * len(layers))()
    outs = []
    for i, L in enumerate(layers):
        X, W = L["X"], L["W"]
        m, n = W.shape
        g = n if L["group_size"] == -1 else L["group_size"]
        o = L.get("out") or {
            "codes": torch.empty((m, n * L["bits"] // 32), dtype=torch.int32, device=dev),
            "scales": torch.empty((m, n // g), dtype=torch.float32, device=dev),
            "zeros": torch.empty((m, n // g), dtype=torch.float32, device=dev),
            "g_idx": torch.empty(n, dtype=torch.int32, device=dev),
            "perm": torch.empty(n, dtype=torch.int32, device=dev),
            "w_hat": torch.empty((m, n), dtype=torch.float32, device=dev) if L.get("want_w_hat") else None}
        outs.append(o)
        j = jobs[i]
        j.X_bf16, j.n_tok, j.ld_x = X.data_ptr(), X.shape[0], X.stride(0)
        j.W_fp16, j.m, j.n = W.data_ptr(), m, n
        j.qp = QParams(int(L["bits"]), int(L["group_size"]), int(bool(L["sym"])))
        j.damp, j.desc_act = float(L["damp"]), int(bool(L["desc_act"]))
        j.codes_out, j.scales_out, j.zeros_out = o["codes"].data_ptr(), o["scales"].data_ptr(), o["zeros"].data_ptr()
        j.g_idx_out, j.perm_out = o["g_idx"].data_ptr(), o["perm"].data_ptr()
        j.W_hat_out = o["w_hat"].data_ptr() if o.get("w_hat") is not None else None
    return jobs, outs


class Pipeline:
    """Contexts kept between batches of layers (gptq_pipeline_*): `widths` maps each input width
    to the largest number of rows its layers have."""

    def __init__(self, widths: dict, device: int = 0, stream: torch.cuda.Stream | None = None):
        self.device = torch.device("cuda", device)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        ws = (ctypes.c_int64 * len(widths))(*[int(w) for w in widths])
        ms = (ctypes.c_int64 * len(widths))(*[int(m) for m in widths.values()])
        h = ctypes.c_void_p()
        _check(lib().gptq_pipeline_create(ctypes.byref(h), ws, ms, len(widths), self.device.index,
                                          ctypes.c_void_p(self.stream.cuda_stream)), "gptq_pipeline_create")
        self._h = h

    def run(self, layers: list) -> list:
        jobs, outs = _jobs(layers, self.device)
        _check(lib().gptq_pipeline_run(self._h, jobs, len(layers)), "gptq_pipeline_run")
        return outs

    def close(self):
        if getattr(self, "_h", None):
            st = lib().gptq_pipeline_destroy(self._h)
            self._h = None
            _check(st, "gptq_pipeline_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


def quantize_layers(layers: list, device: int = 0, stream: torch.cuda.Stream | None = None) -> list:
    """Quantize many layers in one pipelined call (gptq_quantize_layers).  `layers` is a list of
    dicts with X (bf16 [n_tok, n] device tensor; the same tensor object for layers that share an
    input), W (fp16 [m, n]), bits, group_size, sym, damp, desc_act and optional want_w_hat.
    Returns one dict of device outputs per layer (codes, scales, zeros, g_idx, perm, w_hat)."""
    dev = torch.device("cuda", device)
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    jobs, outs = _jobs(layers, dev)
    _check(lib().gptq_quantize_layers(jobs, len(layers), dev.index, ctypes.c_void_p(stream.cuda_stream)),
           "gptq_quantize_layers")
    return outs


def awq_quantize(X: torch.Tensor | None, W: torch.Tensor, s_protect: float = 2.0, bits: int = 4, group_size: int = 128,
                 sym: bool = False, want_w_hat: bool = True, stream: torch.cuda.Stream | None = None) -> dict:
    """AWQ channel scaling plus round-to-nearest (gptq_awq_quantize).  X: bf16 [n_tok, n] device
    tensor (or None: no calibration tokens), W: fp16 [m, n].  Returns device tensors codes,
    scales, zeros, channel_scale and (optionally) w_hat, all in original column order."""
    m, n = W.shape
    dev = W.device
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    g = n if group_size == -1 else group_size
    out = {"codes": torch.empty((m, n * bits // 32), dtype=torch.int32, device=dev),
           "scales": torch.empty((m, n // g), dtype=torch.float32, device=dev),
           "zeros": torch.empty((m, n // g), dtype=torch.float32, device=dev),
           "channel_scale": torch.empty(n, dtype=torch.float32, device=dev),
           "w_hat": torch.empty((m, n), dtype=torch.float32, device=dev) if want_w_hat else None}
    ws = torch.empty(int(lib().gptq_awq_workspace_bytes(n)), dtype=torch.uint8, device=dev)
    n_tok, ld = (0, n) if X is None else (X.shape[0], X.stride(0))
    qp = QParams(int(bits), int(group_size), int(bool(sym)))
    _check(lib().gptq_awq_quantize(_ptr(X), n_tok, ld, _ptr(W), m, n, float(s_protect), qp, _ptr(out["codes"]),
                                   _ptr(out["scales"]), _ptr(out["zeros"]), _ptr(out["channel_scale"]),
                                   _ptr(out["w_hat"]), _ptr(ws), ws.numel(), dev.index,
                                   ctypes.c_void_p(stream.cuda_stream)), "gptq_awq_quantize")
    return out


def rtn_quantize(W: torch.Tensor, bits: int = 8, group_size: int = -1, sym: bool = True, clip_ratio: float = 1.0,
                 channel_scale: torch.Tensor | None = None, want_w_hat: bool = True,
                 stream: torch.cuda.Stream | None = None) -> dict:
    """Round-to-nearest with a clipped range (gptq_rtn_quantize; the page's INT8 LinearQuantizer
    is bits 8, per-channel, symmetric, clip_ratio 0.99).  W: fp16 [m, n]; channel_scale: fp32 [n]
    or None.  Returns device tensors codes, scales, zeros, channel_scale (where one was given) and
    (optionally) w_hat, in original column order."""
    m, n = W.shape
    dev = W.device
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    g = n if group_size == -1 else group_size
    out = {"codes": torch.empty((m, n * bits // 32), dtype=torch.int32, device=dev),
           "scales": torch.empty((m, n // g), dtype=torch.float32, device=dev),
           "zeros": torch.empty((m, n // g), dtype=torch.float32, device=dev),
           "w_hat": torch.empty((m, n), dtype=torch.float32, device=dev) if want_w_hat else None}
    if channel_scale is not None:
        out["channel_scale"] = channel_scale
    qp = QParams(int(bits), int(group_size), int(bool(sym)))
    _check(lib().gptq_rtn_quantize(_ptr(W), m, n, qp, float(clip_ratio), _ptr(channel_scale), _ptr(out["codes"]),
                                   _ptr(out["scales"]), _ptr(out["zeros"]), _ptr(out["w_hat"]), dev.index,
                                   ctypes.c_void_p(stream.cuda_stream)), "gptq_rtn_quantize")
    return out


def activation_convert(Y: torch.Tensor, act: int = 1, want_bf16: bool = True, want_fp16: bool = True,
                       stream: torch.cuda.Stream | None = None):
    """x = act(y) (0 identity, 1 ReLU) of an fp32 or bf16 device tensor, as bf16 and fp16 copies
    (gptq_activation_convert)."""
    if Y.dtype not in (torch.float32, torch.bfloat16) or not Y.is_contiguous():
        raise ValueError("Y must be a contiguous fp32 or bf16 device tensor")
    dev = Y.device
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    xb = torch.empty(Y.shape, dtype=torch.bfloat16, device=dev) if want_bf16 else None
    xh = torch.empty(Y.shape, dtype=torch.float16, device=dev) if want_fp16 else None
    _check(lib().gptq_activation_convert(_ptr(Y), int(Y.dtype == torch.bfloat16), Y.numel(), int(act), _ptr(xb),
                                         _ptr(xh), dev.index, ctypes.c_void_p(stream.cuda_stream)),
           "gptq_activation_convert")
    return xb, xh


def _sequential_context(contexts: dict | None, n: int, m: int, dev: torch.device,
                        stream: torch.cuda.Stream) -> "GPTQContext":
    """A context of width n for at least m rows on this stream: kept in `contexts` when given."""
    if contexts is None:
        return GPTQContext(n, m, dev.index, stream)
    key = (n, dev.index, stream.cuda_stream)
    ctx = contexts.get(key)
    if ctx is not None and ctx.m_max < m:
        ctx.close()
        ctx = None
    if ctx is None:
        ctx = GPTQContext(n, m, dev.index, stream)
        contexts[key] = ctx
    return ctx


def close_contexts(contexts: dict) -> None:
    """Close the contexts that quantize_sequential kept in `contexts`."""
    for ctx in contexts.values():
        ctx.close()
    contexts.clear()


def quantize_sequential(X0: torch.Tensor, layers: list, act: int = 1, stream: torch.cuda.Stream | None = None,
                        keep_hessian: bool = False, contexts: dict | None = None) -> list:
    """Sequential quantization of a stack of linear layers ("GPTQ算法原理深度解析" §2.1: the error
    of a layer reaches the next one through its input).  X0: bf16 [N, n0] calibration inputs of
    layer 0; layers: dicts with W (fp16 [m_l, n_l], n_{l+1} = m_l), bits, group_size, sym, damp,
    desc_act.  Layer l is calibrated on X_l; X_{l+1} = act(X_l W16_l^T), the product taken with
    layer l's quantized weights (gptq_dequant_matmul on the fp16 copy of X_l).  Every step runs in
    the library's kernels; this function only sequences the calls.  Returns, per layer, its
    outputs (codes, scales, zeros, g_idx, perm), its calibration inputs X (bf16) and X16 (the
    fp16 copy its product reads), and with keep_hessian its H (fp32 [n, n]).  contexts: an optional
    dict in which the contexts (one per layer width and stream) stay between calls, so that repeated
    calls skip their creation (workspace allocation, the factorization's graph); the caller closes
    them with close_contexts.  Without it, each layer's context is created and closed here."""
    dev = X0.device
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    xb = X0
    _, xh = activation_convert(X0, act=0, want_bf16=False, stream=stream)
    res = []
    for li, L in enumerate(layers):
        W = L["W"]
        m, n = W.shape
        if xb.shape[1] != n:
            raise ValueError(f"layer {li}: {n} inputs, but the previous layer gives {xb.shape[1]}")
        ctx = _sequential_context(contexts, n, m, dev, stream)
        try:
            ctx.reset()
            ctx.accumulate_hessian(xb)
            H = ctx.get_hessian()[0] if keep_hessian else None
            perm = ctx.prepare(L["damp"], L["desc_act"])
            out = ctx.quantize_layer(W, L["bits"], L["group_size"], L["sym"], want_w_hat=False)
            ctx.synchronize()
        finally:
            if contexts is None:
                ctx.close()
        out = dict(out, perm=perm, X=xb, X16=xh, H=H)
        res.append(out)
        if li + 1 < len(layers):
            Y = dequant_matmul(xh, out["codes"], out["scales"], out["zeros"], perm, L["bits"], L["group_size"],
                               stream=stream)
            xb, xh = activation_convert(Y, act=act, stream=stream)
    return res
